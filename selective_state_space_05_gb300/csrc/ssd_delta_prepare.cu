// The gated delta rule's first launch in fp32: what each chunk needs of its keys,
// queries and gates and not of a state, for all chunks at once.
//
// One CTA of four warps per (chunk, head, batch row):
//   - G, the running sum of g in 64 bits, kept as two floats, so that the decays
//     e^(G_i - G_j) of late tokens do not lose bits to strong earlier ones;
//   - k k^T and q k^T on the tensor cores (lower triangles);
//   - T = (I + N diag(beta))^-1 in fp32: the two 16 x 16 blocks of the diagonal by
//     substitution, a column a lane, then the one below them as -T_11 A_10 T_00.
// T and P are written as bf16 terms, the vectors as fp32.  Bound by the latency of
// the substitution and of the block products in one CTA, of which four or so share an
// SM: 600 chunks of 72 columns in 14.6 us, a twenty-fifth of the call.
#include <math.h>

#include "ssd_delta.cuh"

namespace ssd {
namespace delta {

constexpr int kPrepThreads = 128;

// dst = sgn a b for 16 x 16 blocks in fp32 (row strides LD); 2 x 2 outputs a thread.
template <int LD>
__device__ __forceinline__ void block_product(float* dst, const float* a, const float* b, float sgn,
                                              int tid) {
  if (tid < 64) {
    const int r = tid / 8 * 2, c = tid % 8 * 2;
    float s00 = 0.f, s01 = 0.f, s10 = 0.f, s11 = 0.f;
#pragma unroll 8
    for (int k = 0; k < 16; ++k) {
      const float x0 = a[r * LD + k], x1 = a[(r + 1) * LD + k];
      const float y0 = b[k * LD + c], y1 = b[k * LD + c + 1];
      s00 = fmaf(x0, y0, s00);
      s01 = fmaf(x0, y1, s01);
      s10 = fmaf(x1, y0, s10);
      s11 = fmaf(x1, y1, s11);
    }
    dst[r * LD + c] = sgn * s00;
    dst[r * LD + c + 1] = sgn * s01;
    dst[(r + 1) * LD + c] = sgn * s10;
    dst[(r + 1) * LD + c + 1] = sgn * s11;
  }
}

template <int KP>
__global__ void __launch_bounds__(kPrepThreads) prepare_kernel(const Args a) {
  using M = Mode<float>;
  constexpr int C = M::C, NT = M::NT, TI = M::TI;
  static_assert(C == 32, "a token a lane, two blocks a side");
  constexpr int LD = C + 2;                    // of the fp32 matrices
  constexpr uint32_t kPlane = C * KP * 2;
  extern __shared__ __align__(16) unsigned char smem[];
  float* const vec = reinterpret_cast<float*>(smem);                   // kVecs * C + 4
  unsigned char* const tk = smem + (vec_floats<C>() * 4 + 127) / 128 * 128;
  unsigned char* const tq = tk + TI * kPlane;
  // after the products the tiles' memory holds A, T and a scratch block
  float* const A = reinterpret_cast<float*>(tk);
  float* const Tm = A + C * LD;
  float* const Y = Tm + C * LD;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t id = blockIdx.x;               // (b H + h) nc + c
  const int c = (int)(id % a.nc), h = (int)(id / a.nc % a.H), b = (int)(id / a.nc / a.H);
  const int kg = h / (a.H / a.G);
  const int64_t t0 = (int64_t)c * C;
  const int rows = (int)(a.L - t0 < C ? a.L - t0 : C);
  load_tile<KP, C>(saddr(tk), kPlane,
                   static_cast<const float*>(a.k) + toff(a.sk, b, t0) + (int64_t)kg * a.K, a.sk.t, rows,
                   a.K, a.wide_k, tid, kPrepThreads);
  load_tile<KP, C>(saddr(tq), kPlane,
                   static_cast<const float*>(a.q) + toff(a.sq, b, t0) + (int64_t)kg * a.K, a.sq.t, rows,
                   a.K, a.wide_q, tid, kPrepThreads);
  if (warp == 0) {   // the vectors: a token a lane
    const int i = lane;
    const int64_t t = t0 + i;
    float g = 0.f, be = 0.f;
    int sg = 0;   // resets so far
    if (t < a.L) {
      const int64_t at = ((int64_t)b * a.L + t) * a.H + h;
      g = a.g[at];
      be = a.beta[at];
      if (g < kReset) {
        g = 0.f;
        sg = 1;
      }
      if (a.seq && t > 0) {
        const int32_t* q = a.seq + (int64_t)b * a.L + t;
        if (q[0] != q[-1]) sg = 1;
      }
    }
    double G = (double)g;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const double v = __shfl_up_sync(0xffffffffu, G, off);
      const int n = __shfl_up_sync(0xffffffffu, sg, off);
      if (lane >= off) {
        G += v;
        sg += n;
      }
    }
    const double total = __shfl_sync(0xffffffffu, G, 31);
    const int segs = __shfl_sync(0xffffffffu, sg, 31);
    const float hi = (float)G;
    vec[kGam * C + i] = sg == 0 ? expf(hi) : 0.f;
    vec[kOnto * C + i] = sg == segs ? expf((float)(total - G)) : 0.f;
    vec[kBeta * C + i] = be;
    vec[kRead * C + i] = -vec[kGam * C + i];
    vec[kWrite * C + i] = be * vec[kOnto * C + i];
    vec[kGhi * C + i] = hi;
    vec[kGlo * C + i] = (float)(G - (double)hi);
    vec[kSeg * C + i] = (float)sg;
    if (lane == 0) vec[kVecs * C] = segs == 0 ? expf((float)total) : 0.f;
  }
  __syncthreads();
  float* const gvec = a.vec + id * vec_floats<C>();
  for (int i = tid; i < kVecs * C + 1; i += kPrepThreads) gvec[i] = vec[i];

  // lower triangles of k k^T and q k^T: warp w the rows 16 w ..
  constexpr int NTC = C / 8;
  float kk[NTC][4], qk[NTC][4];
  zero(kk);
  zero(qk);
  if (warp < C / 16) {
    for (int ks = 0; ks < KP / 16; ++ks) {
      uint32_t ak[TI][4], aq[TI][4];
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        ldsm(ak[i], block_at<KP>(saddr(tk) + i * kPlane, warp * 16, ks * 16, lane));
        ldsm(aq[i], block_at<KP>(saddr(tq) + i * kPlane, warp * 16, ks * 16, lane));
      }
#pragma unroll
      for (int n = 0; n < NTC / 2; ++n)
        if (n <= warp) {
          const uint32_t at = blockn_at<KP>(saddr(tk), n * 16, ks * 16, lane);
          mma_pair<TI, TI, false>(kk[2 * n], kk[2 * n + 1], ak, at, kPlane);
          mma_pair<TI, TI, false>(qk[2 * n], qk[2 * n + 1], aq, at, kPlane);
        }
    }
  }
  __syncthreads();   // the tiles' memory is A's from here
  bf16* const gP = a.P + id * NT * C * C;
  if (warp < C / 16) {
#pragma unroll
    for (int n = 0; n < NTC; ++n) {
      if (n / 2 > warp) continue;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int i = warp * 16 + (lane >> 2) + 8 * r, j = n * 8 + (lane & 3) * 2;
        float p[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool near = i >= j + e && vec[kSeg * C + i] == vec[kSeg * C + j + e];
          const float d = near ? expf((vec[kGhi * C + i] - vec[kGhi * C + j + e]) +
                                      (vec[kGlo * C + i] - vec[kGlo * C + j + e]))
                               : 0.f;
          p[e] = near ? a.scale * qk[n][2 * r + e] * d : 0.f;
          A[i * LD + j + e] = near && i > j + e ? kk[n][2 * r + e] * d * vec[kBeta * C + j + e] : 0.f;
        }
        uint32_t w[NT];
        split2<NT>(p[0], p[1], w);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          *reinterpret_cast<uint32_t*>(gP + (t * C + i) * C + j) = w[t];
      }
    }
  }
  __syncthreads();
  // T: the diagonal's 16 x 16 blocks
  if (warp < C / 16 && lane < 16) {
    const int r0 = warp * 16;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == lane ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < i; ++j) s = fmaf(-A[(r0 + i) * LD + r0 + j], x[j], s);
      x[i] = s;
      Tm[(r0 + i) * LD + r0 + lane] = s;
    }
  }
  __syncthreads();
  // the block below them (what is above them is not read)
  block_product<LD>(Y + 16 * LD, A + 16 * LD, Tm, 1.f, tid);
  __syncthreads();
  block_product<LD>(Tm + 16 * LD, Tm + 16 * LD + 16, Y + 16 * LD, -1.f, tid);
  __syncthreads();
  bf16* const gT = a.T + id * NT * C * C;
  for (int o = tid; o < C * C / 2; o += kPrepThreads) {
    const int i = o / (C / 2), j = o % (C / 2) * 2;
    if (j / 16 > i / 16) continue;
    uint32_t w[NT];
    split2<NT>(Tm[i * LD + j], Tm[i * LD + j + 1], w);
#pragma unroll
    for (int t = 0; t < NT; ++t) *reinterpret_cast<uint32_t*>(gT + (t * C + i) * C + j) = w[t];
  }
}

template <int KP>
cudaError_t prepare(const Args& a, cudaStream_t st) {
  using M = Mode<float>;
  constexpr int C = M::C;
  const int tiles = 2 * M::TI * C * KP * 2, mats = 3 * C * (C + 2) * 4;
  const int smem = (vec_floats<C>() * 4 + 127) / 128 * 128 + (tiles > mats ? tiles : mats);
  cudaError_t e = cudaFuncSetAttribute(prepare_kernel<KP>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t n = (int64_t)a.B * a.H * a.nc;
  prepare_kernel<KP><<<(unsigned)n, kPrepThreads, smem, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_prepare(const Args& a, cudaStream_t st) {
  return a.KP == 64 ? prepare<64>(a, st) : prepare<128>(a, st);
}

}  // namespace delta
}  // namespace ssd
