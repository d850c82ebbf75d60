// The gated delta rule's backward within each chunk in fp32, all chunks at once.  With
// the state S0 before a chunk, dS after it, x and dy (kept as terms) and dout:
//   dq0 = scale e^G (do S0),  dk0 = -e^G (dy S0),  w0 = e^(G_C - G) (x dS)
//   dp = do x^T,  da = dy x^T,   P, N the chunk's scores and keys' products (with
//   their decays D, computed again),  H = dp P - da N
//   M1 = scale D dp beta,  M2 = -D da beta (strictly lower)
//   dq = dq0 + M1 k,   dk = dk0 + M2 k + beta w0 + M1^T q + M2^T k
//   dbeta_j = k_j w0_j + sum_i H_ij
//   dg_t = e^(G_C) <dS, S0> + sum_{i>=t} (q_i dq0_i + k_i dk0_i)
//          + sum_{j<t} beta_j k_j w0_j + sum_{i>=t>j} H_ij beta_j
// The last line takes each pair of tokens around t once (all of its terms are
// what they are in the recurrence: no sums over the chunk that cancel).
//
// One CTA of eight warps per (chunk, head, batch row).  The [C, dstate] results
// stay in accumulators, 16 rows and a part of the columns a warp; the sums over
// headdim run in tiles of 32 channels that arrive by cp.async one ahead.  600 chunks
// of 64 channels and 72 columns take 72 us: each CTA's products are few, and its loads
// and sums wait for each other.
#include "ssd_delta.cuh"

namespace ssd {
namespace delta {

constexpr int kGradThreads = 256, kVT = 32;   // kVT: channels a tile

template <int KP>
struct GradSmem {
  using M = Mode<float>;
  static constexpr int C = M::C, RG = C / 16, CG = 8 / RG;   // row and column groups of warps
  static constexpr uint32_t kPlane = C * KP * 2;             // K, Q
  static constexpr uint32_t kTok = C * kVT * 2;              // dout, x, dy
  static constexpr uint32_t kState = kVT * KP * 2;           // S0, dS
  static constexpr uint32_t kMat = C * C * 2;                // M1, M2
  static constexpr uint32_t k = 0, q = M::TI * kPlane, vec = 2 * M::TI * kPlane,
                            red = vec + (vec_floats<C>() * 4 + 127) / 128 * 128,
                            st = red + ((2 * CG * C + C + 16) * 4 + 127) / 128 * 128;
  // a stage
  static constexpr uint32_t d = 0, x = M::TI * kTok, y = x + M::NT * kTok, s0 = y + M::NT * kTok,
                            ds = s0 + M::NT * kState, stage = ds + M::NT * kState;
  // after the tiles, in their memory
  static constexpr uint32_t m1 = st, m2 = m1 + M::NT * kMat, hm = m2 + M::NT * kMat,
                            end = hm + C * (C + 1) * 4;
  static constexpr uint32_t total = st + 2 * stage > end ? st + 2 * stage : end;
};

template <int KP>
__device__ __forceinline__ void load_channels(const Args& a, uint32_t st, int b, int h, int64_t id,
                                              int64_t t0, int rows, int v0, int tid) {
  using S = GradSmem<KP>;
  constexpr int C = S::C, NT = S::M::NT;
  const int cols = a.V - v0 < kVT ? a.V - v0 : kVT, pad = a.VP - v0 < kVT ? a.VP - v0 : kVT;
  load_tile<kVT, C>(st + S::d, S::kTok,
                    static_cast<const float*>(a.dout) + toff(a.sdo, b, t0) + (int64_t)h * a.V + v0,
                    a.sdo.t, rows, cols, a.wide_do, tid, kGradThreads);
  load_planes<kVT, C, NT>(st + S::x, S::kTok, a.X + id * NT * C * a.VP + v0, a.VP,
                          (int64_t)C * a.VP, C, pad, tid, kGradThreads);
  load_planes<kVT, C, NT>(st + S::y, S::kTok, a.dY + id * NT * C * a.VP + v0, a.VP,
                          (int64_t)C * a.VP, C, pad, tid, kGradThreads);
  load_planes<KP, kVT, NT>(st + S::s0, S::kState, a.S0 + (id * NT * a.VP + v0) * KP, KP,
                           (int64_t)a.VP * KP, pad, KP, tid, kGradThreads);
  load_planes<KP, kVT, NT>(st + S::ds, S::kState, a.dS + (id * NT * a.VP + v0) * KP, KP,
                           (int64_t)a.VP * KP, pad, KP, tid, kGradThreads);
}

// A row's pair of columns in a result of `cols` columns.
__device__ __forceinline__ void put2(float* row, int c, int cols, bool pairs, float x, float y) {
  if (pairs && c + 1 < cols) {
    *reinterpret_cast<float2*>(row + c) = make_float2(x, y);
  } else {
    if (c < cols) row[c] = x;
    if (c + 1 < cols) row[c + 1] = y;
  }
}

template <int KP>
__global__ void __launch_bounds__(kGradThreads) grads_kernel(const Args a) {
  using S = GradSmem<KP>;
  constexpr int C = S::C, NT = S::M::NT, TI = S::M::TI, RG = S::RG, CG = S::CG;
  constexpr int NW = KP / CG / 16;                     // 16-column blocks of a warp's results
  static_assert(RG <= CG, "a warp has one 16-column block of the pair matrices: cg's");
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3, rg = warp % RG, cg = warp / RG;
  const int64_t id = blockIdx.x;
  const int c = (int)(id % a.nc), h = (int)(id / a.nc % a.H), b = (int)(id / a.nc / a.H);
  const int kg = h / (a.H / a.G);
  const int64_t t0 = (int64_t)c * C;
  const int rows = (int)(a.L - t0 < C ? a.L - t0 : C);
  const uint32_t base = saddr(smem);
  float* const vec = reinterpret_cast<float*>(smem + S::vec);
  float* const rd = reinterpret_cast<float*>(smem + S::red);   // [CG][C], then w0's, <dS, S0>
  float* const wd = rd + CG * C;
  float* const acc = wd + CG * C;
  float* const part = acc + C;

  load_tile<KP, C>(base + S::k, S::kPlane,
                   static_cast<const float*>(a.k) + toff(a.sk, b, t0) + (int64_t)kg * a.K, a.sk.t, rows,
                   a.K, a.wide_k, tid, kGradThreads);
  load_tile<KP, C>(base + S::q, S::kPlane,
                   static_cast<const float*>(a.q) + toff(a.sq, b, t0) + (int64_t)kg * a.K, a.sq.t, rows,
                   a.K, a.wide_q, tid, kGradThreads);
  for (int i = tid; i < vec_floats<C>() / 4; i += kGradThreads)
    cp16(base + S::vec + i * 16, a.vec + id * vec_floats<C>() + i * 4, 16);
  load_channels<KP>(a, base + S::st, b, h, id, t0, rows, 0, tid);
  cp_commit();

  float dq[2 * NW][4], dk[2 * NW][4], w0[2 * NW][4], dp[2][4], da[2][4];
  zero(dq);
  zero(dk);
  zero(w0);
  zero(dp);
  zero(da);
  float inner = 0.f;
  const int tiles = (a.VP + kVT - 1) / kVT;
  for (int v = 0; v < tiles; ++v) {
    const uint32_t at = S::st + (v & 1) * S::stage, st = base + at;
    cp_wait<0>();
    __syncthreads();
    if (v + 1 < tiles)
      load_channels<KP>(a, base + S::st + ((v + 1) & 1) * S::stage, b, h, id, t0, rows,
                        (v + 1) * kVT, tid);
    cp_commit();
#pragma unroll
    for (int ks = 0; ks < kVT / 16; ++ks) {
      uint32_t fd[TI][4], fx[NT][4], fy[NT][4];
#pragma unroll
      for (int i = 0; i < TI; ++i)
        ldsm(fd[i], block_at<kVT>(st + S::d + i * S::kTok, rg * 16, ks * 16, lane));
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        ldsm(fx[i], block_at<kVT>(st + S::x + i * S::kTok, rg * 16, ks * 16, lane));
        ldsm(fy[i], block_at<kVT>(st + S::y + i * S::kTok, rg * 16, ks * 16, lane));
      }
#pragma unroll
      for (int n = 0; n < NW; ++n) {
        const int col = (cg * NW + n) * 16;
        const uint32_t s0 = block_at<KP>(st + S::s0, ks * 16, col, lane);
        mma_apart<TI, NT, true>(dq[2 * n], dq[2 * n + 1], fd, s0, S::kState);
        mma_apart<NT, NT, true>(dk[2 * n], dk[2 * n + 1], fy, s0, S::kState);
        mma_apart<NT, NT, true>(w0[2 * n], w0[2 * n + 1], fx,
                               block_at<KP>(st + S::ds, ks * 16, col, lane), S::kState);
      }
      if (cg <= rg) {
        const uint32_t xt = blockn_at<kVT>(st + S::x, cg * 16, ks * 16, lane);
        mma_apart<TI, NT, false>(dp[0], dp[1], fd, xt, S::kTok);
        mma_apart<NT, NT, false>(da[0], da[1], fy, xt, S::kTok);
      }
    }
    for (int i = tid; i < kVT * KP / 2; i += kGradThreads) {
      const int r = i / (KP / 2), col = i % (KP / 2) * 2;
      const float2 x = tile_pair<KP, NT>(smem + at + S::s0, S::kState, r, col);
      const float2 y = tile_pair<KP, NT>(smem + at + S::ds, S::kState, r, col);
      inner = fmaf(x.x, y.x, fmaf(x.y, y.y, inner));
    }
  }

  // the decays of the reads and the write, and their sums over dstate with q and k
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int i = rg * 16 + g + 8 * r;
    const float gam = vec[kGam * C + i], onto = vec[kOnto * C + i], be = vec[kBeta * C + i];
    float sr = 0.f, sw = 0.f;
#pragma unroll
    for (int n = 0; n < 2 * NW; ++n) {
      const int col = cg * NW * 16 + n * 8 + t * 2;
      const float2 qv = tile_pair<KP, TI>(smem + S::q, S::kPlane, i, col);
      const float2 kv = tile_pair<KP, TI>(smem + S::k, S::kPlane, i, col);
      float *x = &dq[n][2 * r], *y = &dk[n][2 * r], *z = &w0[n][2 * r];
      x[0] *= a.scale * gam;
      x[1] *= a.scale * gam;
      y[0] *= -gam;
      y[1] *= -gam;
      z[0] *= onto;
      z[1] *= onto;
      sr += qv.x * x[0] + qv.y * x[1] + kv.x * y[0] + kv.y * y[1];
      sw += kv.x * z[0] + kv.y * z[1];
      y[0] = fmaf(be, z[0], y[0]);
      y[1] = fmaf(be, z[1], y[1]);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      sr += __shfl_xor_sync(0xffffffffu, sr, o);
      sw += __shfl_xor_sync(0xffffffffu, sw, o);
    }
    if (t == 0) {
      rd[cg * C + i] = sr;
      wd[cg * C + i] = sw;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, o);
  if (lane == 0) part[warp] = inner;

  // the chunk's scores again, for the pairs' gradients
  float qk[2][4], kk[2][4];
  zero(qk);
  zero(kk);
#pragma unroll 2
  for (int ks = 0; ks < KP / 16; ++ks) {
    uint32_t fq[TI][4], fk[TI][4];
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      ldsm(fq[i], block_at<KP>(base + S::q + i * S::kPlane, rg * 16, ks * 16, lane));
      ldsm(fk[i], block_at<KP>(base + S::k + i * S::kPlane, rg * 16, ks * 16, lane));
    }
    if (cg <= rg) {
      const uint32_t kt = blockn_at<KP>(base + S::k, cg * 16, ks * 16, lane);
      mma_apart<TI, TI, false>(qk[0], qk[1], fq, kt, S::kPlane);
      mma_apart<TI, TI, false>(kk[0], kk[1], fk, kt, S::kPlane);
    }
  }
  __syncthreads();   // the tiles' memory is M1's, M2's and H's from here
  float* const hm = reinterpret_cast<float*>(smem + S::hm);
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    if (cg > rg) continue;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = rg * 16 + g + 8 * r, j = cg * 16 + n * 8 + t * 2;
      float u1[2], u2[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool near = i >= j + e && vec[kSeg * C + i] == vec[kSeg * C + j + e];
        const float d = near ? expf((vec[kGhi * C + i] - vec[kGhi * C + j + e]) +
                                    (vec[kGlo * C + i] - vec[kGlo * C + j + e]))
                             : 0.f;
        const float strict = i > j + e ? d : 0.f, be = vec[kBeta * C + j + e];
        const float x = dp[n][2 * r + e], y = da[n][2 * r + e];
        hm[i * (C + 1) + j + e] = x * (a.scale * d * qk[n][2 * r + e]) - y * (strict * kk[n][2 * r + e]);
        u1[e] = a.scale * d * x * be;
        u2[e] = -strict * y * be;
      }
      uint32_t w[NT];
      split2<NT>(u1[0], u1[1], w);
      const uint32_t at = tile_at<C>(i, j >> 3) + (j & 7) * 2;
#pragma unroll
      for (int m = 0; m < NT; ++m)
        *reinterpret_cast<uint32_t*>(smem + S::m1 + m * S::kMat + at) = w[m];
      split2<NT>(u2[0], u2[1], w);
#pragma unroll
      for (int m = 0; m < NT; ++m)
        *reinterpret_cast<uint32_t*>(smem + S::m2 + m * S::kMat + at) = w[m];
    }
  }
  __syncthreads();
#pragma unroll
  for (int ks = 0; ks < C / 16; ++ks) {
    if (ks <= rg) {   // rows rg of M1 and M2, keys ks
      uint32_t f1[NT][4], f2[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        ldsm(f1[i], block_at<C>(base + S::m1 + i * S::kMat, rg * 16, ks * 16, lane));
        ldsm(f2[i], block_at<C>(base + S::m2 + i * S::kMat, rg * 16, ks * 16, lane));
      }
#pragma unroll
      for (int n = 0; n < NW; ++n) {
        const uint32_t kt = block_at<KP>(base + S::k, ks * 16, (cg * NW + n) * 16, lane);
        mma_apart<NT, TI, true>(dq[2 * n], dq[2 * n + 1], f1, kt, S::kPlane);
        mma_apart<NT, TI, true>(dk[2 * n], dk[2 * n + 1], f2, kt, S::kPlane);
      }
    }
    if (ks >= rg) {   // columns rg, queries and keys ks
      uint32_t f1[NT][4], f2[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        a_from_t(f1[i], block_at<C>(base + S::m1 + i * S::kMat, ks * 16, rg * 16, lane));
        a_from_t(f2[i], block_at<C>(base + S::m2 + i * S::kMat, ks * 16, rg * 16, lane));
      }
#pragma unroll
      for (int n = 0; n < NW; ++n) {
        const int col = (cg * NW + n) * 16;
        mma_apart<NT, TI, true>(dk[2 * n], dk[2 * n + 1], f1,
                               block_at<KP>(base + S::q, ks * 16, col, lane), S::kPlane);
        mma_apart<NT, TI, true>(dk[2 * n], dk[2 * n + 1], f2,
                               block_at<KP>(base + S::k, ks * 16, col, lane), S::kPlane);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int i = rg * 16 + g + 8 * r;
    if (i >= rows) continue;
    const int64_t tok = (int64_t)b * a.L + t0 + i;
#pragma unroll
    for (int n = 0; n < 2 * NW; ++n) {
      const int col = cg * NW * 16 + n * 8 + t * 2;
      const bool pairs = a.K % 2 == 0;
      if (a.dq_part) {
        const int64_t row = (tok * a.H + h) * a.K;
        put2(a.dq_part + row, col, a.K, pairs, dq[n][2 * r], dq[n][2 * r + 1]);
        put2(a.dk_part + row, col, a.K, pairs, dk[n][2 * r], dk[n][2 * r + 1]);
      } else {
        const int64_t row = (tok * a.G + kg) * a.K;
        put2(static_cast<float*>(a.dq) + row, col, a.K, pairs, dq[n][2 * r], dq[n][2 * r + 1]);
        put2(static_cast<float*>(a.dk) + row, col, a.K, pairs, dk[n][2 * r], dk[n][2 * r + 1]);
      }
    }
  }
  // beta's gradient, and H summed over the rows from t on for each column
  if (tid < C) {
    const int j = tid;
    const float be = vec[kBeta * C + j];
    float w = 0.f, run = 0.f;
#pragma unroll
    for (int p = 0; p < CG; ++p) w += wd[p * C + j];
    for (int i = C - 1; i > j; --i) {
      run += hm[i * (C + 1) + j];
      hm[i * (C + 1) + j] = run * be;
    }
    run += hm[j * (C + 1) + j];
    if (j < rows) a.dbeta[((int64_t)b * a.L + t0 + j) * a.H + h] = w + run;
    wd[j] = w * be;
    float x = 0.f;
#pragma unroll
    for (int p = 0; p < CG; ++p) x += rd[p * C + j];
    acc[j] = x;
  }
  __syncthreads();
  if (tid < rows) {
    float x = 0.f, y = 0.f, z = 0.f, total = 0.f;
    for (int j = 0; j < tid; ++j) {
      x += hm[tid * (C + 1) + j];
      y += wd[j];
    }
    for (int i = C - 1; i >= tid; --i) z += acc[i];
#pragma unroll
    for (int w = 0; w < kGradThreads / 32; ++w) total += part[w];
    // (a state that starts anew at t leaves t nothing to decay: all four are 0)
    a.dg[((int64_t)b * a.L + t0 + tid) * a.H + h] = vec[kVecs * C] * total + z + y + x;
  }
}

// Heads that share queries and keys: their gradients' sum, in the heads' order.
template <typename T>
__global__ void __launch_bounds__(256)
    group_sum_kernel(const float* __restrict__ dq, const float* __restrict__ dk, int64_t rows,
                     int R, int K, T* __restrict__ oq, T* __restrict__ ok) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * K;
       i += (int64_t)gridDim.x * 256) {
    const int64_t at = i / K * R * K + i % K;
    float x = 0.f, y = 0.f;
    for (int r = 0; r < R; ++r) {
      x += dq[at + (int64_t)r * K];
      y += dk[at + (int64_t)r * K];
    }
    oq[i] = from_f<T>(x);
    ok[i] = from_f<T>(y);
  }
}

template <typename T>
cudaError_t launch_group_sum(const Args& a, cudaStream_t st) {
  const int64_t rows = (int64_t)a.B * a.L * a.G, ctas = (rows * a.K + 255) / 256;
  group_sum_kernel<T><<<(unsigned)(ctas < 65536 ? ctas : 65536), 256, 0, st>>>(
      a.dq_part, a.dk_part, rows, a.H / a.G, a.K, static_cast<T*>(a.dq), static_cast<T*>(a.dk));
  return cudaGetLastError();
}
template cudaError_t launch_group_sum<bf16>(const Args&, cudaStream_t);
template cudaError_t launch_group_sum<float>(const Args&, cudaStream_t);

template <int KP>
cudaError_t grads(const Args& a, cudaStream_t st) {
  using S = GradSmem<KP>;
  cudaError_t e = cudaFuncSetAttribute(grads_kernel<KP>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, S::total);
  if (e != cudaSuccess) return e;
  const int64_t n = (int64_t)a.B * a.H * a.nc;
  grads_kernel<KP><<<(unsigned)n, kGradThreads, S::total, st>>>(a);
  if (a.dq_part) return launch_group_sum<float>(a, st);
  return cudaGetLastError();
}

cudaError_t launch_grads(const Args& a, cudaStream_t st) {
  return a.KP == 64 ? grads<64>(a, st) : grads<128>(a, st);
}

}  // namespace delta
}  // namespace ssd
