// The gated delta rule's forward in fp32 over the chunks of each (batch row, head),
// one after another, with the state in registers.
//
// A warp owns 16 rows of S (16 of the headdim channels) as mma accumulators, and
// everything in a chunk is computed transposed, [channels, tokens], so that each
// result is the next product's A operand in the same registers:
//   y = v - e^G (S k),   x = y T^T,   u = beta x,   o = scale e^G (S q) + u P^T,
//   S = e^(G_C) S + (e^(G_C - G) u) K
// The CTA's warps share the chunk's K, Q, T and P in shared memory, which four more
// warps load and split one chunk ahead; one barrier a chunk is all that the warps
// wait for each other.  The write into S is summed apart from S and added with one
// rounding, since the tensor cores' sums truncate and S lives for many chunks.
// Bound by a warp's own chain of products, six mma a pair of factors.  24 sequences of 25
// chunks, 64 channels and 72 columns take 144 us, 5.8 a chunk: with fewer heads than SMs a
// CTA has one warp with rows, so that 96 SMs have one such warp each, and one quadrant of
// the four at work.  Columns past dstate are not multiplied, which is 3/8 of them there.
#include "ssd_delta_seq.cuh"

namespace ssd {
namespace delta {

template <int KP>
struct FwdSmem {
  using M = Mode<float>;
  static constexpr int C = M::C;
  static constexpr uint32_t kPlane = C * KP * 2;        // of K and Q
  static constexpr uint32_t kMat = C * C * 2;           // of T and P
  static constexpr uint32_t vpitch(int nw) { return nw * 16 * sizeof(float) + 16; }
  static constexpr uint32_t kVec = (vec_floats<C>() * 4 + 15) / 16 * 16;
  static constexpr uint32_t k = 0, q = M::TI * kPlane, t = 2 * M::TI * kPlane,
                            p = t + M::NT * kMat, vec = p + M::NT * kMat, v = vec + kVec;
  static constexpr uint32_t stage(int nw) { return (v + C * vpitch(nw) + 127) / 128 * 128; }
  // a warp's results on their way out: C rows of 16 values
  static constexpr uint32_t opitch = 16 * sizeof(float) + 16;
  static constexpr uint32_t total(int nw) { return 2 * stage(nw) + nw * C * opitch; }
};

// One chunk's operands into a stage.
template <int KP>
__device__ __forceinline__ void load_chunk(const Args& a, uint32_t st, int b, int h, int kg, int c,
                                           int v0, int nw, int tid, int nth) {
  using S = FwdSmem<KP>;
  constexpr int C = S::C, NT = S::M::NT;
  const int64_t t0 = (int64_t)c * C;
  const int rows = (int)(a.L - t0 < C ? a.L - t0 : C);
  const int64_t id = ((int64_t)b * a.H + h) * a.nc + c;
  load_tile<KP, C>(st + S::k, S::kPlane,
                   static_cast<const float*>(a.k) + toff(a.sk, b, t0) + (int64_t)kg * a.K, a.sk.t, rows,
                   a.K, a.wide_k, tid, nth);
  if (a.out)
    load_tile<KP, C>(st + S::q, S::kPlane,
                     static_cast<const float*>(a.q) + toff(a.sq, b, t0) + (int64_t)kg * a.K, a.sq.t,
                     rows, a.K, a.wide_q, tid, nth);
  load_planes<C, C, NT>(st + S::t, S::kMat, a.T + id * NT * C * C, C, C * C, C, C, tid, nth);
  if (a.out)
    load_planes<C, C, NT>(st + S::p, S::kMat, a.P + id * NT * C * C, C, C * C, C, C, tid, nth);
  const float* gv = a.vec + id * vec_floats<C>();
  for (int i = tid; i < vec_floats<C>() / 4; i += nth) cp16(st + S::vec + i * 16, gv + i * 4, 16);
  // v: rows of nw * 16 channels from v0 on
  const float* src = static_cast<const float*>(a.v) + toff(a.sv, b, t0) + (int64_t)h * a.V + v0;
  constexpr int E = 16 / sizeof(float);
  const int cols = a.V - v0 < nw * 16 ? a.V - v0 : nw * 16, units = nw * 16 / E;
  for (int i = tid; i < C * units; i += nth) {
    const int r = i / units, u = i % units;
    const uint32_t at = st + S::v + r * S::vpitch(nw) + u * 16;
    const float* p = src + r * a.sv.t + u * E;
    if (a.wide_v) {
      const bool in = r < rows && u * E < cols;
      cp16(at, in ? p : src, in ? 16 : 0);
    } else {
      union {
        float e[E];
        uint4 w;
      } x;
      x.w = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (r < rows && u * E + j < cols) x.e[j] = p[j];
      sts16(at, x.w.x, x.w.y, x.w.z, x.w.w);
    }
  }
}

template <int KP>
__global__ void __launch_bounds__(256) forward_kernel(const Args a) {
  using S = FwdSmem<KP>;
  constexpr int C = S::C, NT = S::M::NT, TI = S::M::TI, NC = C / 8, NK = KP / 8;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nw = (blockDim.x >> 5) - kLoadWarps;   // those with rows
  // the loading threads: the warps behind them
  const int ltid = tid - nw * 32;
  constexpr int nth = kLoadWarps * 32;
  const int g = lane >> 2, t = lane & 3;
  const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H, kg = h / (a.H / a.G);
  const int v0 = blockIdx.y * nw * 16, vw = v0 + warp * 16;   // the CTA's, the warp's channels
  const uint32_t base = saddr(smem);
  unsigned char* const obuf = smem + 2 * S::stage(nw) + warp * C * S::opitch;

  float s[NK][4];
  read_state<KP>(s, a.init ? a.init + (int64_t)bh * a.V * a.K : nullptr, vw, a.V, a.K, lane);
  if (ltid >= 0) load_chunk<KP>(a, base, b, h, kg, 0, v0, nw, ltid, nth);
  cp_commit();
  for (int c = 0; c < a.nc; ++c) {
    const uint32_t off = (c & 1) * S::stage(nw);
    cp_wait<0>();
    __syncthreads();   // the chunk is there, and all warps are done with the one before
    if (ltid >= 0 && c + 1 < a.nc)
      load_chunk<KP>(a, base + (S::stage(nw) - off), b, h, kg, c + 1, v0, nw, ltid, nth);
    cp_commit();
    if (warp >= nw) continue;   // (it only loads)
    if (vw >= a.VP) continue;   // (it only helps to load)
    const uint32_t st = base + off;
    const float* vec = reinterpret_cast<const float*>(smem + off + S::vec);
    const int64_t id = (int64_t)bh * a.nc + c;
    const int64_t t0 = (int64_t)c * C;
    const int rows = (int)(a.L - t0 < C ? a.L - t0 : C);
    if (a.S0) store_state<KP, NT>(s, a.S0 + (id * NT * a.VP + vw) * KP, (int64_t)a.VP * KP, lane);

    float y[NC][4], o[NC][4];
    zero(y);
    zero(o);
#pragma unroll
    for (int ks = 0; ks < KP / 16; ++ks) {
      if (ks * 16 >= a.K) break;
      uint32_t f[NT][4];
      a_from<NT>(s[2 * ks], s[2 * ks + 1], f);
#pragma unroll
      for (int n = 0; n < NC / 2; ++n) {
        mma_apart<NT, TI, false>(y[2 * n], y[2 * n + 1], f,
                                blockn_at<KP>(st + S::k, n * 16, ks * 16, lane), S::kPlane);
        if (a.out)
          mma_apart<NT, TI, false>(o[2 * n], o[2 * n + 1], f,
                                  blockn_at<KP>(st + S::q, n * 16, ks * 16, lane), S::kPlane);
      }
    }
    const unsigned char* vt = smem + off + S::v + (warp * 16 + g) * sizeof(float);
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int i = n * 8 + t * 2;
      const float2 gam = ld2(vec + kGam * C + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = to_f(*reinterpret_cast<const float*>(vt + (i + (e & 1)) * S::vpitch(nw) +
                                                         8 * (e >> 1) * sizeof(float)));
        const float ge = e & 1 ? gam.y : gam.x;
        y[n][e] = fmaf(-ge, y[n][e], v);
        o[n][e] *= a.scale * ge;
      }
    }
    float x[NC][4];
    zero(x);
    mma_lower<C, NT>(x, y, st + S::t, lane);
    if (a.X) store_terms<C, NT>(x, obuf, S::opitch, a.X + id * NT * C * a.VP + vw, a.VP,
                                (int64_t)C * a.VP, lane);
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const float2 be = ld2(vec + kBeta * C + n * 8 + t * 2);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[n][e] *= e & 1 ? be.y : be.x;
    }
    if (a.out) {
      mma_lower<C, NT>(o, x, st + S::p, lane);
      store_rows<float, C>(o, obuf, S::opitch,
                       static_cast<float*>(a.out) + (((int64_t)b * a.L + t0) * a.H + h) * a.V + vw,
                       (int64_t)a.H * a.V, rows, a.V - vw, a.wide_out, lane);
    }
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const float2 on = ld2(vec + kOnto * C + n * 8 + t * 2);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[n][e] *= e & 1 ? on.y : on.x;
    }
    uint32_t f[C / 16][NT][4];
#pragma unroll
    for (int ks = 0; ks < C / 16; ++ks) a_from<NT>(x[2 * ks], x[2 * ks + 1], f[ks]);
    const float through = vec[kVecs * C];
#pragma unroll
    for (int n = 0; n < NK / 2; ++n) {
      if (n * 16 >= a.K) break;
      float w[2][4];
      zero(w);
#pragma unroll
      for (int ks = 0; ks < C / 16; ++ks)
        mma_apart<NT, TI, true>(w[0], w[1], f[ks], block_at<KP>(st + S::k, ks * 16, n * 16, lane),
                               S::kPlane);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[2 * n][e] = fmaf(through, s[2 * n][e], w[0][e]);
        s[2 * n + 1][e] = fmaf(through, s[2 * n + 1][e], w[1][e]);
      }
    }
  }
  cp_wait<0>();
  if (a.final && warp < nw && vw < a.VP)
    write_state<KP>(s, a.final + (int64_t)bh * a.V * a.K, vw, a.V, a.K, lane);
}

template <int KP>
cudaError_t forward(const Args& a, cudaStream_t st) {
  using S = FwdSmem<KP>;
  int nw = 0;
  cudaError_t e = warps_for(a, &nw);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(forward_kernel<KP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::total(kRowWarps));
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(a.B * a.H), (unsigned)((a.VP / 16 + nw - 1) / nw));
  forward_kernel<KP><<<grid, (nw + kLoadWarps) * 32, S::total(nw), st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_forward(const Args& a, cudaStream_t st) {
  return a.KP == 64 ? forward<64>(a, st) : forward<128>(a, st);
}

}  // namespace delta
}  // namespace ssd
