// The gated delta rule's backward along the sequence in fp32, last chunk first, with
// the state's gradient dS in registers, transposed as in the forward:
//   dx = beta (do P + e^(G_C - G) (dS k)),   dy = dx T
//   dS <- e^(G_C) dS + (scale e^G do) Q - (e^G dy) K
// dy is the gradient of v.  dS at each chunk's end and dy are kept as terms for
// the chunks' own gradients, which need no order.  Bound as the forward, and as
// fast: 141 us for 24 sequences of 25 chunks.
#include "ssd_delta_seq.cuh"

namespace ssd {
namespace delta {

template <int KP>
struct RevSmem {
  using M = Mode<float>;
  static constexpr int C = M::C;
  static constexpr uint32_t kPlane = C * KP * 2;
  static constexpr uint32_t kMat = C * C * 2;
  static constexpr uint32_t kOut = C * 16 * 2;          // a plane of a warp's 16 columns of dout
  static constexpr uint32_t kVec = (vec_floats<C>() * 4 + 127) / 128 * 128;
  static constexpr uint32_t k = 0, q = M::TI * kPlane, t = 2 * M::TI * kPlane,
                            p = t + M::NT * kMat, vec = p + M::NT * kMat, d = vec + kVec;
  static constexpr uint32_t stage(int nw) { return d + nw * M::TI * kOut; }
  static constexpr uint32_t opitch = 16 * sizeof(float) + 16;
  static constexpr uint32_t total(int nw) { return 2 * stage(nw) + nw * C * opitch; }
};

template <int KP>
__device__ __forceinline__ void load_reverse(const Args& a, uint32_t st, int b, int h, int kg,
                                             int c, int v0, int nw, int tid, int nth) {
  using S = RevSmem<KP>;
  constexpr int C = S::C, NT = S::M::NT;
  const int64_t t0 = (int64_t)c * C;
  const int rows = (int)(a.L - t0 < C ? a.L - t0 : C);
  const int64_t id = ((int64_t)b * a.H + h) * a.nc + c;
  load_tile<KP, C>(st + S::k, S::kPlane,
                   static_cast<const float*>(a.k) + toff(a.sk, b, t0) + (int64_t)kg * a.K, a.sk.t, rows,
                   a.K, a.wide_k, tid, nth);
  load_tile<KP, C>(st + S::q, S::kPlane,
                   static_cast<const float*>(a.q) + toff(a.sq, b, t0) + (int64_t)kg * a.K, a.sq.t, rows,
                   a.K, a.wide_q, tid, nth);
  load_planes<C, C, NT>(st + S::t, S::kMat, a.T + id * NT * C * C, C, C * C, C, C, tid, nth);
  load_planes<C, C, NT>(st + S::p, S::kMat, a.P + id * NT * C * C, C, C * C, C, C, tid, nth);
  const float* gv = a.vec + id * vec_floats<C>();
  for (int i = tid; i < vec_floats<C>() / 4; i += nth) cp16(st + S::vec + i * 16, gv + i * 4, 16);
  const float* src = static_cast<const float*>(a.dout) + toff(a.sdo, b, t0) + (int64_t)h * a.V;
  for (int w = 0; w < nw; ++w) {
    const int v = v0 + w * 16, cols = a.V - v < 16 ? a.V - v : 16;
    load_tile<16, C>(st + S::d + w * S::M::TI * S::kOut, S::kOut, src + (cols > 0 ? v : 0), a.sdo.t,
                     rows, cols > 0 ? cols : 0, a.wide_do, tid, nth);
  }
}

template <int KP>
__global__ void __launch_bounds__(256) reverse_kernel(const Args a) {
  using S = RevSmem<KP>;
  constexpr int C = S::C, NT = S::M::NT, TI = S::M::TI, NC = C / 8, NK = KP / 8;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nw = (blockDim.x >> 5) - kLoadWarps;   // those with rows
  // the loading threads: the warps behind them
  const int ltid = tid - nw * 32;
  constexpr int nth = kLoadWarps * 32;
  const int t = lane & 3;
  const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H, kg = h / (a.H / a.G);
  const int v0 = blockIdx.y * nw * 16, vw = v0 + warp * 16;
  const uint32_t base = saddr(smem);
  unsigned char* const obuf = smem + 2 * S::stage(nw) + warp * C * S::opitch;

  float s[NK][4];
  read_state<KP>(s, a.dfinal ? a.dfinal + (int64_t)bh * a.V * a.K : nullptr, vw, a.V, a.K, lane);
  if (ltid >= 0) load_reverse<KP>(a, base, b, h, kg, a.nc - 1, v0, nw, ltid, nth);
  cp_commit();
  for (int n0 = 0; n0 < a.nc; ++n0) {
    const int c = a.nc - 1 - n0;
    const uint32_t off = (n0 & 1) * S::stage(nw);
    cp_wait<0>();
    __syncthreads();   // the chunk is there, and all warps are done with the one before
    if (ltid >= 0 && c > 0)
      load_reverse<KP>(a, base + (S::stage(nw) - off), b, h, kg, c - 1, v0, nw, ltid, nth);
    cp_commit();
    if (warp >= nw) continue;   // (it only loads)
    if (vw >= a.VP) continue;   // (it only helps to load)
    const uint32_t st = base + off;
    const float* vec = reinterpret_cast<const float*>(smem + off + S::vec);
    const int64_t id = (int64_t)bh * a.nc + c;
    const int64_t t0 = (int64_t)c * C;
    const int rows = (int)(a.L - t0 < C ? a.L - t0 : C);
    store_state<KP, NT>(s, a.dS + (id * NT * a.VP + vw) * KP, (int64_t)a.VP * KP, lane);

    float x[NC][4];
    zero(x);
#pragma unroll
    for (int ks = 0; ks < KP / 16; ++ks) {
      if (ks * 16 >= a.K) break;
      uint32_t f[NT][4];
      a_from<NT>(s[2 * ks], s[2 * ks + 1], f);
#pragma unroll
      for (int n = 0; n < NC / 2; ++n)
        mma_apart<NT, TI, false>(x[2 * n], x[2 * n + 1], f,
                                blockn_at<KP>(st + S::k, n * 16, ks * 16, lane), S::kPlane);
    }
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const float2 on = ld2(vec + kOnto * C + n * 8 + t * 2);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[n][e] *= e & 1 ? on.y : on.x;
    }
    uint32_t d[C / 16][TI][4];   // dout as A operand, [channel, token]
    const uint32_t dt = st + S::d + warp * TI * S::kOut;
#pragma unroll
    for (int ks = 0; ks < C / 16; ++ks) {
#pragma unroll
      for (int i = 0; i < TI; ++i)
        a_from_t(d[ks][i], block_at<16>(dt + i * S::kOut, ks * 16, 0, lane));
#pragma unroll
      for (int n = 0; n <= ks; ++n)
        mma_apart<TI, NT, true>(x[2 * n], x[2 * n + 1], d[ks],
                               block_at<C>(st + S::p, ks * 16, n * 16, lane), S::kMat);
    }
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const float2 be = ld2(vec + kBeta * C + n * 8 + t * 2);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[n][e] *= e & 1 ? be.y : be.x;
    }
    float y[NC][4];
    zero(y);
#pragma unroll
    for (int ks = 0; ks < C / 16; ++ks) {
      uint32_t f[NT][4];
      a_from<NT>(x[2 * ks], x[2 * ks + 1], f);
#pragma unroll
      for (int n = 0; n <= ks; ++n)
        mma_apart<NT, NT, true>(y[2 * n], y[2 * n + 1], f,
                               block_at<C>(st + S::t, ks * 16, n * 16, lane), S::kMat);
    }
    store_terms<C, NT>(y, obuf, S::opitch, a.dY + id * NT * C * a.VP + vw, a.VP, (int64_t)C * a.VP,
                       lane);
    store_rows<float, C>(y, obuf, S::opitch,
                     static_cast<float*>(a.dv) + (((int64_t)b * a.L + t0) * a.H + h) * a.V + vw,
                     (int64_t)a.H * a.V, rows, a.V - vw, a.wide_dv, lane);
    uint32_t fq[C / 16][NT][4], fk[C / 16][NT][4];
#pragma unroll
    for (int ks = 0; ks < C / 16; ++ks) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {   // the left and right eight tokens
        const float2 gam = ld2(vec + kGam * C + (2 * ks + j) * 8 + t * 2);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float u0 = 0.f, u1 = 0.f;
#pragma unroll
          for (int i = TI - 1; i >= 0; --i) {
            u0 += lo_of(d[ks][i][2 * j + r]);
            u1 += hi_of(d[ks][i][2 * j + r]);
          }
          uint32_t w[NT];
          split2<NT>(u0 * (a.scale * gam.x), u1 * (a.scale * gam.y), w);
#pragma unroll
          for (int i = 0; i < NT; ++i) fq[ks][i][2 * j + r] = w[i];
          split2<NT>(-gam.x * y[2 * ks + j][2 * r], -gam.y * y[2 * ks + j][2 * r + 1], w);
#pragma unroll
          for (int i = 0; i < NT; ++i) fk[ks][i][2 * j + r] = w[i];
        }
      }
    }
    const float through = vec[kVecs * C];
#pragma unroll
    for (int n = 0; n < NK / 2; ++n) {
      if (n * 16 >= a.K) break;
      float w[2][4];
      zero(w);
#pragma unroll
      for (int ks = 0; ks < C / 16; ++ks) {
        mma_apart<NT, TI, true>(w[0], w[1], fq[ks], block_at<KP>(st + S::q, ks * 16, n * 16, lane),
                               S::kPlane);
        mma_apart<NT, TI, true>(w[0], w[1], fk[ks], block_at<KP>(st + S::k, ks * 16, n * 16, lane),
                               S::kPlane);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[2 * n][e] = fmaf(through, s[2 * n][e], w[0][e]);
        s[2 * n + 1][e] = fmaf(through, s[2 * n + 1][e], w[1][e]);
      }
    }
  }
  cp_wait<0>();
  if (a.dinit && warp < nw && vw < a.VP)
    write_state<KP>(s, a.dinit + (int64_t)bh * a.V * a.K, vw, a.V, a.K, lane);
}

template <int KP>
cudaError_t reverse(const Args& a, cudaStream_t st) {
  using S = RevSmem<KP>;
  int nw = 0;
  cudaError_t e = warps_for(a, &nw);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(reverse_kernel<KP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::total(kRowWarps));
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(a.B * a.H), (unsigned)((a.VP / 16 + nw - 1) / nw));
  reverse_kernel<KP><<<grid, (nw + kLoadWarps) * 32, S::total(nw), st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_reverse(const Args& a, cudaStream_t st) {
  return a.KP == 64 ? reverse<64>(a, st) : reverse<128>(a, st);
}

}  // namespace delta
}  // namespace ssd
