// The gated delta rule's backward within each chunk on tcgen05 (its formulas:
// ssd_delta_grads.cu), one CTA per SM, a chunk of a (head, batch row) after another.
// With the state S0 before the chunk, dS after it, x and dY as terms (hi, lo) and dout:
//   D5 = [K; Q] K^T                                lanes: rows of K, of Q
//   D3 = [dYhi; do] [Xhi; Xlo]^T,  D3lo = dYlo Xhi^T  lanes: rows of dY, of do
//   from them, a row a thread:  M2 = -D da beta, M1 = scale D dp beta as terms, and H
//   D1 = S0^T [dY | do],  D2 = dS^T [Xhi | Xlo]    lanes: dstate
//   D4 = K^T [M2; M1]^T,  its first half += Q^T M1 + K^T M2
//   dq = scale e^G D1[do] + D4[1],  dk = -e^G D1[dY] + beta e^(G_C - G) D2 + D4[0]
// A tile serves in the order in which it is needed: K and Q by tokens and by
// dstate, M by rows and by columns; the terms of B's rows stand side by side in N, so
// that an MMA has 128 columns.  S0, dS, x and dY (192 KB a chunk and head) come once,
// K, Q and dout too: dS takes S0's place in shared memory as soon as D1 is done and
// the warps have S0 in registers for <S0, dS>; every buffer's next load starts as soon
// as it is free.  Sums over dstate run over the lanes with shuffles.
// Bound by the sixteen warps' own work, phase after phase (7000 instructions a chunk
// and quadrant): 10240 chunks in 502 us, 5.5 TB/s.  Before the next chunk's D3 was computed
// while this one's tokens are summed, for which D1 and D3 change places in TMEM, it took
// 682; a CTA a chunk, with S0 read again for <S0, dS>, 752.
#include "ssd_delta_tc.cuh"
#include "ssd_row.cuh"

namespace ssd {
namespace delta {
namespace grd {

constexpr int kWarps = 16, kMmaWarp = 16, kLoadWarp = 17;
constexpr int kThreads = 20 * 32;   // (two idle, for the register split)
// TMEM columns: D3lo, D2 (Xhi, Xlo), D5; D1 (dY, do) and D3 (then D4), which change places
// with each chunk: D3 is computed as soon as the D1 before it is read
constexpr uint32_t kD3lo = 128, kD2 = 192, kD5 = 448;
__device__ __forceinline__ uint32_t d1_at(int it) { return it & 1 ? 320 : 0; }
__device__ __forceinline__ uint32_t d3_at(int it) { return it & 1 ? 0 : 320; }
constexpr int kHPitch = 65;

template <int KP>
struct Smem {
  static constexpr uint32_t kHalf = 2 * kTile;
  unsigned char kq[KP / 64][2][kTile];   // 64 dstate columns: K, Q
  unsigned char q[2][kTile];             // a channel half: dYlo
  union {
    unsigned char m[2][2][kTile];        // a term: M2, M1 (D3lo reads what stands there too)
    unsigned char out[2][KP / 64][kTile];   // then dq, dk
  };
  unsigned char x[2][2][kTile];          // a channel half: Xhi, Xlo
  unsigned char s[2][KP / 8][128][16];   // a term, 8 dstate columns, 128 channels: S0, then dS
  union {
    unsigned char p[2][2][kTile];        // a channel half: dYhi, do
    float h[128][kHPitch];               // then H's rows of dY, of do
  };
  alignas(16) float vec[2][vec_floats<kC>()];
  float rd[4][kC], wd[4][kC];            // sums over a quarter of dstate: reads, write
  float around[kWarps][kC], total[kC], inner[kWarps];
  // copies that have landed, products done, and what the warps are through with
  uint64_t kq_full, x_full, p_full, q_full, s_full, ds_full;
  uint64_t d3_done, d1_done, d2_done, d4_done, drain_bar;
  uint64_t m_ready, s_read, s_free, kq_free, p_free, out_free, d1_read, d_free;
  uint32_t tmem;
  volatile int gave_up;
};

__device__ int g_status;
std::atomic<bool> g_launched{false};

// D (+)= A B over STEPS steps of 16 along K: descriptors and what a step adds.
template <int STEPS>
__device__ __forceinline__ void chain(uint32_t d, uint64_t a, uint32_t sa, uint64_t b, uint32_t sb,
                                      uint32_t idesc, bool fresh) {
#pragma unroll
  for (int ks = 0; ks < STEPS; ++ks)
    tc::mma_ss(d, a + ks * sa, b + ks * sb, idesc, !(fresh && ks == 0));
}
// Asks for bytes (a multiple of 16) to be brought to the L2.
__device__ __forceinline__ void prefetch(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
// Sums of 16 values each over the warp's lanes: lane l gets value l / 2's.
__device__ __forceinline__ float lane_sums(float (&x)[16], int lane) {
#pragma unroll
  for (int n = 8; n >= 1; n >>= 1) {   // lanes exchange half of what they still have
    const bool up = lane & (2 * n);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? x[i] : x[i + n], keep = up ? x[i + n] : x[i];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2 * n);
    }
  }
  return x[0] + __shfl_xor_sync(0xffffffffu, x[0], 1);
}

template <int KP>
__global__ void __launch_bounds__(kThreads, 1)
    tc_grads_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap md, const __grid_constant__ CUtensorMap moq,
                    const __grid_constant__ CUtensorMap mok, const int tma_out,
                    const __grid_constant__ Args a) {
  extern __shared__ unsigned char raw[];
  using S = Smem<KP>;
  S& s = *reinterpret_cast<S*>(raw + ((1024 - (saddr(raw) & 1023)) & 1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunks = a.B * a.H * a.nc;         // (each has 64 KB and more: an int)
  const int blocks = a.VP / 128;               // of 128 channels
  if (warp == kMmaWarp) tc::tmem_alloc(&s.tmem, 512);
  if (tid == 0) {
    uint64_t* const one[] = {&s.kq_full, &s.x_full,  &s.p_full,  &s.q_full,
                             &s.s_full,  &s.ds_full, &s.d3_done, &s.d1_done,
                             &s.d2_done, &s.d4_done, &s.out_free, &s.drain_bar};
    for (uint64_t* p : one) tc::mbar_init(p, 1);
    uint64_t* const all[] = {&s.m_ready, &s.s_read,  &s.s_free, &s.kq_free,
                             &s.p_free,  &s.d1_read, &s.d_free};
    for (uint64_t* p : all) tc::mbar_init(p, kWarps);
    tc::mbar_fence_init();
    s.gave_up = 0;
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s.tmem;
  auto W = [&](uint64_t* bar, uint32_t parity) { wait_for(bar, parity, &s.gave_up, &g_status); };
  // halves of 64 channels in block v
  auto halves = [&](int v) { return a.V - v * 128 > 64 ? 2 : 1; };

  if (warp >= kMmaWarp) {
    SSD_SETREG("dec", "64");
    if (warp == kLoadWarp) {
      auto bulk = [&](void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
        tc::bulk_load(dst, src, bytes, bar);
      };
      auto stop = [&] { return __any_sync(0xffffffffu, s.gave_up) != 0; };
      auto block_of = [&](const bf16* planes, int id, int v) {
        return reinterpret_cast<const unsigned char*>(planes) +
               ((int64_t)id * blocks + v) * sizeof(s.s);
      };
      // how many of each have been asked for
      int kqs = 0, xs = 0, ps = 0, qs = 0, ss = 0, dss = 0, it = 0, n = 0;
      for (int id = blockIdx.x; id < chunks && !stop(); id += gridDim.x, ++it) {
        const int c = id % a.nc, h = id / a.nc % a.H, b = id / a.nc / a.H;
        const int kg = h / (a.H / a.G);
        // a state's planes of block v
        auto state = [&](const bf16* planes, int v, uint64_t* bar) {
          tc::mbar_arrive_expect_tx(bar, sizeof(s.s));
          bulk(s.s, block_of(planes, id, v), sizeof(s.s), bar);
        };
        for (int v = 0; v < blocks; ++v, ++n) {
          const int nh = halves(v);
          const int64_t tile = (int64_t)id * 2 * (a.VP / 64) + v * 2;   // the first term's
          const unsigned char* y = reinterpret_cast<const unsigned char*>(a.dY) + tile * kTile;
          const unsigned char* x = reinterpret_cast<const unsigned char*>(a.X) + tile * kTile;
          const int64_t next = (int64_t)(a.VP / 64) * kTile;
          if (n > 0) {
            W(&s.d2_done, (n - 1) & 1);
            W(&s.s_free, (n - 1) & 1);
          }
          if (stop()) break;
          if (tc::elect_one()) {
            tc::mbar_arrive_expect_tx(&s.x_full, nh * 2 * kTile);
            for (int i = 0; i < nh; ++i) {
              bulk(s.x[i][0], x + i * kTile, kTile, &s.x_full);
              bulk(s.x[i][1], x + next + i * kTile, kTile, &s.x_full);
            }
            state(a.S0, v, &s.s_full);
            prefetch(block_of(a.dS, id, v), sizeof(s.s));
          }
          __syncwarp();
          ++xs;
          ++ss;
          if (v == 0) {
            if (it > 0) {
              W(&s.d4_done, (it - 1) & 1);
              W(&s.kq_free, (it - 1) & 1);
            }
            if (stop()) break;
            if (tc::elect_one()) {
              tc::mbar_arrive_expect_tx(&s.kq_full, KP / 64 * 2 * kTile + vec_floats<kC>() * 4);
              for (int i = 0; i < KP / 64; ++i) {
                tc::tma_load_4d(s.kq[i][0], &mk, &s.kq_full, i * 64, kg, c * kC, b);
                tc::tma_load_4d(s.kq[i][1], &mq, &s.kq_full, i * 64, kg, c * kC, b);
              }
              bulk(s.vec[it & 1], a.vec + (int64_t)id * vec_floats<kC>(), vec_floats<kC>() * 4,
                   &s.kq_full);
            }
            __syncwarp();
            ++kqs;
            if (it > 0) W(&s.p_free, (it - 1) & 1);
          } else {
            W(&s.d1_done, (n - 1) & 1);
          }
          if (stop()) break;
          if (tc::elect_one()) {
            tc::mbar_arrive_expect_tx(&s.p_full, nh * 2 * kTile);
            for (int i = 0; i < nh; ++i) {
              bulk(s.p[i][0], y + i * kTile, kTile, &s.p_full);
              tc::tma_load_4d(s.p[i][1], &md, &s.p_full, v * 128 + i * 64, h, c * kC, b);
            }
          }
          __syncwarp();
          ++ps;
          if (tc::elect_one()) {   // (D1 of the block before is done)
            tc::mbar_arrive_expect_tx(&s.q_full, nh * kTile);
            for (int i = 0; i < nh; ++i) bulk(s.q[i], y + next + i * kTile, kTile, &s.q_full);
          }
          __syncwarp();
          ++qs;
          W(&s.d1_done, n & 1);
          W(&s.s_read, n & 1);
          if (stop()) break;
          if (tc::elect_one()) state(a.dS, v, &s.ds_full);
          __syncwarp();
          ++dss;
        }
      }
      // every copy has landed before the CTA ends
      auto last = [&](uint64_t* bar, int count) {
        if (count) drain(bar, (count - 1) & 1, &g_status);
      };
      last(&s.kq_full, kqs);
      last(&s.x_full, xs);
      last(&s.p_full, ps);
      last(&s.q_full, qs);
      last(&s.s_full, ss);
      last(&s.ds_full, dss);
    } else if (warp == kMmaWarp) {
      constexpr uint32_t kk128 = tc::idesc_bf16(128, 128, false, false);
      constexpr uint32_t kk64 = tc::idesc_bf16(128, 64, false, false);
      constexpr uint32_t mk128 = tc::idesc_bf16(128, 128, true, false);
      constexpr uint32_t mk64 = tc::idesc_bf16(128, 64, true, false);
      constexpr uint32_t mm64 = tc::idesc_bf16(128, 64, true, true);
      constexpr uint32_t tile = kTile >> 4;
      // (with 64 dstate columns the MMA's upper 64 rows are not read)
      constexpr uint32_t mkq = KP == 128 ? S::kHalf : 0;
      const uint64_t dk = tc::sdesc_sw128(saddr(s.kq[0][0]), 16, 1024);
      const uint64_t dkm = tc::sdesc_sw128(saddr(s.kq[0][0]), mkq, 1024);
      const uint64_t dp = tc::sdesc_sw128(saddr(s.p[0][0]), 16, 1024);
      const uint64_t dq = tc::sdesc_sw128(saddr(s.q[0]), 16, 1024);
      const uint64_t dx = tc::sdesc_sw128(saddr(s.x[0][0]), 16, 1024);
      const uint64_t dsm = sdesc_rows(saddr(s.s));
      const uint64_t dm = tc::sdesc_sw128(saddr(s.m[0][0]), 16, 1024);
      const uint64_t dmm = tc::sdesc_sw128(saddr(s.m[0][0]), kTile, 1024);
      constexpr uint32_t term = (KP / 8) * 2048 >> 4;   // a state's second term
      auto stop = [&] { return __any_sync(0xffffffffu, s.gave_up) != 0; };
      int it = 0, n = 0;
      for (int id = blockIdx.x; id < chunks && !stop(); id += gridDim.x, ++it) {
        W(&s.kq_full, it & 1);
        if (stop()) break;
        tc::fence_after_sync();
        if (tc::elect_one()) {   // (D5 was read before M was ready)
          for (int i = 0; i < KP / 64; ++i)
            chain<4>(tmem + kD5, dk + i * 2 * tile, 2, dk + i * 2 * tile, 2, kk64, i == 0);
        }
        __syncwarp();
        const uint32_t kD1 = d1_at(it), kD3 = d3_at(it);
        if (it > 0) W(&s.d1_read, (it - 1) & 1);
        for (int v = 0; v < blocks; ++v, ++n) {
          const uint32_t ph = n & 1;
          const int nh = halves(v);
          W(&s.x_full, ph);
          W(&s.p_full, ph);
          W(&s.q_full, ph);
          if (stop()) break;
          tc::fence_after_sync();
          if (tc::elect_one()) {
            for (int i = 0; i < nh; ++i) {   // (D3lo's lanes from 64 on are of what lies behind)
              const uint32_t at = i * 2 * tile;
              const bool fresh = v == 0 && i == 0;
              chain<4>(tmem + kD3, dp + at, 2, dx + at, 2, kk128, fresh);
              chain<4>(tmem + kD3lo, dq + i * tile, 2, dx + at, 2, kk64, fresh);
            }
            tc::mma_commit(&s.d3_done);
          }
          __syncwarp();
          if (v == 0 && it > 0) W(&s.d_free, (it - 1) & 1);
          W(&s.s_full, ph);
          if (stop()) break;
          tc::fence_after_sync();
          if (tc::elect_one()) {
            for (int i = 0; i < nh; ++i) {   // 64 channels: 4 steps of 16 rows
              const uint32_t at = i * 2 * tile, rows = i * (64 * 16 >> 4);
              const bool fresh = v == 0 && i == 0;
              chain<4>(tmem + kD1, dsm + term + rows, 16, dp + at, 2, mk128, fresh);
              chain<4>(tmem + kD1, dsm + rows, 16, dq + i * tile, 2, mk64, false);
              chain<4>(tmem + kD1, dsm + rows, 16, dp + at, 2, mk128, false);
            }
            tc::mma_commit(&s.d1_done);
          }
          __syncwarp();
          if (v + 1 == blocks) {   // (while dS comes)
            W(&s.m_ready, it & 1);
            if (stop()) break;
            tc::fence_after_sync();
            if (tc::elect_one()) {
              for (int t = 1; t >= 0; --t)
                chain<4>(tmem + kD3, dkm, 128, dm + t * 2 * tile, 2, mk128, t == 1);
              for (int t = 1; t >= 0; --t) {
                chain<4>(tmem + kD3, dkm + tile, 128, dmm + t * 2 * tile + tile, 128, mm64, false);
                chain<4>(tmem + kD3, dkm, 128, dmm + t * 2 * tile, 128, mm64, false);
              }
              tc::mma_commit(&s.d4_done);
            }
            __syncwarp();
          }
          W(&s.ds_full, ph);
          if (stop()) break;
          tc::fence_after_sync();
          if (tc::elect_one()) {
            for (int i = 0; i < nh; ++i) {
              const uint32_t at = i * 2 * tile, rows = i * (64 * 16 >> 4);
              const bool fresh = v == 0 && i == 0;
              chain<4>(tmem + kD2, dsm + rows, 16, dx + at, 2, mk128, fresh);
              chain<4>(tmem + kD2, dsm + term + rows, 16, dx + at, 2, mk64, false);
            }
            tc::mma_commit(&s.d2_done);
          }
          __syncwarp();
        }
      }
      if (tc::elect_one()) tc::mma_commit(&s.drain_bar);
      __syncwarp();
      drain(&s.drain_bar, 0, &g_status);
    }
  } else {
    SSD_SETREG("inc", "104");
    const int qr = warp & 3, part = warp >> 2, row = qr * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)qr << 21);
    const int t0 = part * 16;
    int it = 0, n = 0;
    for (int id = blockIdx.x; id < chunks; id += gridDim.x, ++it, ++n) {
      const int c = id % a.nc, h = id / a.nc % a.H, b = id / a.nc / a.H;
      const int kg = h / (a.H / a.G);
      const int rows = (int)(a.L - (int64_t)c * kC < kC ? a.L - (int64_t)c * kC : kC);
      const float* const vec = s.vec[it & 1];
      const uint32_t kD1 = d1_at(it), kD3 = d3_at(it);
      // <S0, dS>: a thread's pieces of S0 wait in registers for dS, which takes its place
      constexpr int pieces = KP / 8 * 128, mine = pieces / (kWarps * 32);
      float inner = 0.f, s0[mine][8];
      const uint4* const planes = reinterpret_cast<const uint4*>(s.s);
      auto take_state = [&] {
        W(&s.s_full, n & 1);
#pragma unroll
        for (int k = 0; k < mine; ++k) {
          const uint4 x = planes[tid + k * kWarps * 32], y = planes[pieces + tid + k * kWarps * 32];
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s0[k][2 * e] = lo_of(xs[e]) + lo_of(ys[e]);
            s0[k][2 * e + 1] = hi_of(xs[e]) + hi_of(ys[e]);
          }
        }
        warp_arrive(&s.s_read, lane);
      };
      auto inner_with = [&] {
        W(&s.ds_full, n & 1);
#pragma unroll
        for (int k = 0; k < mine; ++k) {
          const uint4 x = planes[tid + k * kWarps * 32], y = planes[pieces + tid + k * kWarps * 32];
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            inner = fmaf(s0[k][2 * e], lo_of(xs[e]) + lo_of(ys[e]), inner);
            inner = fmaf(s0[k][2 * e + 1], hi_of(xs[e]) + hi_of(ys[e]), inner);
          }
        }
        warp_arrive(&s.s_free, lane);
      };
      for (int v = 0; v + 1 < blocks; ++v, ++n) {
        take_state();
        inner_with();
      }
      take_state();

      // ---------------- the pairs: row of dY (lanes 0-63) or of do, 16 columns
      W(&s.kq_full, it & 1);
      W(&s.d3_done, n & 1);
      tc::fence_after_sync();
      {
        const int i = row & 63;
        const bool reads = row >= 64;   // a query's row
        float u[16], hh[16];
        {
          uint32_t r[16], r2[16];
          tc::tmem_ld16(lanes + kD3 + t0, r);
          tc::tmem_ld16(lanes + kD3 + 64 + t0, r2);
          tc::tmem_ld_wait_regs(r);
          tc::tmem_ld_wait_regs(r2);
#pragma unroll
          for (int e = 0; e < 16; ++e) u[e] = __uint_as_float(r[e]) + __uint_as_float(r2[e]);
          if (!reads) {   // (a warp's rows are of one kind)
            tc::tmem_ld16(lanes + kD3lo + t0, r);
            tc::tmem_ld_wait_regs(r);
#pragma unroll
            for (int e = 0; e < 16; ++e) u[e] += __uint_as_float(r[e]);
          }
          tc::tmem_ld16(lanes + kD5 + t0, r);
          tc::tmem_ld_wait_regs(r);
          const float neg = __int_as_float(0xff800000), f = reads ? a.scale : -1.f;
          const float hi = vec[kGhi * kC + i], lo = vec[kGlo * kC + i], sg = vec[kSeg * kC + i];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int j = t0 + 4 * q;
            const float4 h4 = *reinterpret_cast<const float4*>(vec + kGhi * kC + j);
            const float4 l4 = *reinterpret_cast<const float4*>(vec + kGlo * kC + j);
            const float4 s4 = *reinterpret_cast<const float4*>(vec + kSeg * kC + j);
            const float hj[4] = {h4.x, h4.y, h4.z, h4.w}, lj[4] = {l4.x, l4.y, l4.z, l4.w};
            const float sj[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool near = sj[e] == sg && (i > j + e || (reads && i == j + e));
              const float d = ex2(near ? (hi - hj[e]) + (lo - lj[e]) : neg) * f;
              const int n = 4 * q + e;
              u[n] = near ? u[n] * d : 0.f;
              hh[n] = near ? u[n] * __uint_as_float(r[n]) : 0.f;
            }
          }
          scale_by(u, vec + kBeta * kC + t0);
          two_terms(u, r);
          tc::fence_before_sync();
          W(&s.d1_done, n & 1);   // dY's and do's memory is H's from here
          if (it > 0) W(&s.out_free, (it - 1) & 1);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            unsigned char* p = s.m[0][reads ? 1 : 0] + tile_at<64>(i, (t0 >> 3) + e);
            *reinterpret_cast<uint4*>(p) =
                make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
            *reinterpret_cast<uint4*>(p + 2 * kTile) =
                make_uint4(r[8 + 4 * e], r[9 + 4 * e], r[10 + 4 * e], r[11 + 4 * e]);
          }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) s.h[row][t0 + e] = hh[e];
      }
      tc::fence_proxy_async_smem();
      warp_arrive(&s.m_ready, lane);
      inner_with();
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, o);
      named_sync(1, kWarps * 32);   // H is whole
      if (lane == 0) s.inner[warp] = inner;
      {
        // four columns of H a warp, rows over the lanes: sums over the rows from each on
        float a0 = 0.f, a1 = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = warp * 4 + e;
          float x0 = s.h[lane][j] + s.h[64 + lane][j], x1 = s.h[32 + lane][j] + s.h[96 + lane][j];
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const float y0 = __shfl_down_sync(0xffffffffu, x0, o);
            const float y1 = __shfl_down_sync(0xffffffffu, x1, o);
            if (lane + o < 32) {
              x0 += y0;
              x1 += y1;
            }
          }
          x0 += __shfl_sync(0xffffffffu, x1, 0);
          const float be = vec[kBeta * kC + j];
          if (lane == 0) s.total[j] = x0;
          if (lane > j) a0 = fmaf(x0, be, a0);
          if (lane + 32 > j) a1 = fmaf(x1, be, a1);
        }
        s.around[warp][lane] = a0;
        s.around[warp][lane + 32] = a1;
      }
      tc::fence_proxy_async_smem();
      warp_arrive(&s.p_free, lane);
      // ---------------- the tokens: dstate row `row`, 16 tokens
      const bool live = row < KP;
      float x[16], y[16];
      uint32_t r[16], kv[8], qv[8];
      {
        const int kc = row & (KP - 1);   // (the upper lanes are copies with 64 columns)
        const unsigned char* base = s.kq[kc >> 6][0] + (kc & 7) * 2;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const unsigned char* p0 = base + tile_at<64>(t0 + 2 * e, (kc & 63) >> 3);
          const unsigned char* p1 = base + tile_at<64>(t0 + 2 * e + 1, (kc & 63) >> 3);
          kv[e] = *reinterpret_cast<const uint16_t*>(p0) |
                  (uint32_t)*reinterpret_cast<const uint16_t*>(p1) << 16;
          qv[e] = *reinterpret_cast<const uint16_t*>(p0 + kTile) |
                  (uint32_t)*reinterpret_cast<const uint16_t*>(p1 + kTile) << 16;
        }
      }
      warp_arrive(&s.kq_free, lane);
      float dq[16], dk[16];
      tc::fence_after_sync();
      tc::tmem_ld16(lanes + kD1 + 64 + t0, r);
      tc::tmem_ld_wait_regs(r);
#pragma unroll
      for (int e = 0; e < 16; ++e) dq[e] = __uint_as_float(r[e]) * a.scale;
      scale_by(dq, vec + kGam * kC + t0);
      tc::tmem_ld16(lanes + kD1 + t0, r);
      tc::tmem_ld_wait_regs(r);
#pragma unroll
      for (int e = 0; e < 16; ++e) dk[e] = __uint_as_float(r[e]);
      tc::fence_before_sync();
      warp_arrive(&s.d1_read, lane);
      scale_by(dk, vec + kRead * kC + t0);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[2 * e] = live ? lo_of(qv[e]) * dq[2 * e] + lo_of(kv[e]) * dk[2 * e] : 0.f;
        x[2 * e + 1] = live ? hi_of(qv[e]) * dq[2 * e + 1] + hi_of(kv[e]) * dk[2 * e + 1] : 0.f;
      }
      {
        const float sum = lane_sums(x, lane);
        if ((lane & 1) == 0) s.rd[qr][t0 + (lane >> 1)] = sum;
      }
      W(&s.d2_done, n & 1);
      W(&s.d4_done, it & 1);
      tc::fence_after_sync();
      tc::tmem_ld16(lanes + kD2 + t0, r);
      tc::tmem_ld_wait_regs(r);
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = __uint_as_float(r[e]);
      tc::tmem_ld16(lanes + kD2 + 64 + t0, r);
      tc::tmem_ld_wait_regs(r);
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] += __uint_as_float(r[e]);
      scale_by(y, vec + kOnto * kC + t0);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[2 * e] = live ? lo_of(kv[e]) * y[2 * e] : 0.f;
        x[2 * e + 1] = live ? hi_of(kv[e]) * y[2 * e + 1] : 0.f;
      }
      {
        const float sum = lane_sums(x, lane);
        if ((lane & 1) == 0) s.wd[qr][t0 + (lane >> 1)] = sum;
      }
      scale_by(y, vec + kBeta * kC + t0);
      tc::tmem_ld16(lanes + kD3 + t0, r);
      tc::tmem_ld_wait_regs(r);
#pragma unroll
      for (int e = 0; e < 16; ++e) dk[e] += y[e] + __uint_as_float(r[e]);
      tc::tmem_ld16(lanes + kD3 + 64 + t0, r);
      tc::tmem_ld_wait_regs(r);
#pragma unroll
      for (int e = 0; e < 16; ++e) dq[e] += __uint_as_float(r[e]);
      tc::fence_before_sync();
      warp_arrive(&s.d_free, lane);
      const int64_t tok = (int64_t)b * a.L + (int64_t)c * kC + t0;
      if (tma_out) {   // M's memory is dq's and dk's now
        if (live) {
          unsigned char* base = s.out[0][row >> 6] + (row & 7) * 2;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            unsigned char* p = base + tile_at<64>(t0 + e, (row & 63) >> 3);
            *reinterpret_cast<bf16*>(p) = __float2bfloat16_rn(dq[e]);
            *reinterpret_cast<bf16*>(p + (KP / 64) * kTile) = __float2bfloat16_rn(dk[e]);
          }
        }
        tc::fence_proxy_async_smem();
      } else if (row < a.K) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (t0 + e >= rows) break;
          if (a.dq_part) {
            const int64_t at = ((tok + e) * a.H + h) * a.K + row;
            a.dq_part[at] = dq[e];
            a.dk_part[at] = dk[e];
          } else {
            const int64_t at = ((tok + e) * a.G + kg) * a.K + row;
            static_cast<bf16*>(a.dq)[at] = __float2bfloat16_rn(dq[e]);
            static_cast<bf16*>(a.dk)[at] = __float2bfloat16_rn(dk[e]);
          }
        }
      }
      named_sync(1, kWarps * 32);
      if (warp == 0 && tc::elect_one()) {
        if (tma_out && !s.gave_up) {
          for (int k = 0; k < KP / 64; ++k)
            if (k * 64 < a.K) {
              tc::tma_store_4d(&moq, s.out[0][k], k * 64, kg, c * kC, b);
              tc::tma_store_4d(&mok, s.out[1][k], k * 64, kg, c * kC, b);
            }
          tc::bulk_commit();
          tc::bulk_wait_read();
        }
        tc::mbar_arrive(&s.out_free);
      }
      __syncwarp();
      // ---------------- beta's and the decays' gradients: a token a lane of two warps
      if (warp == 1 || warp == 2) {
        const int t = (warp - 1) * 32 + lane;
        float total = 0.f, near = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          total += s.inner[w];
          near += s.around[w][t];
        }
        // sums over the reads from t on and over the writes before t
        auto read = [&](int i) { return s.rd[0][i] + s.rd[1][i] + s.rd[2][i] + s.rd[3][i]; };
        auto put = [&](int i) { return s.wd[0][i] + s.wd[1][i] + s.wd[2][i] + s.wd[3][i]; };
        float r0 = read(lane), r1 = read(lane + 32);
        const float p0 = put(lane), p1 = put(lane + 32);
        float w0 = p0 * vec[kBeta * kC + lane], w1 = p1 * vec[kBeta * kC + lane + 32];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float y0 = __shfl_down_sync(0xffffffffu, r0, o);
          const float y1 = __shfl_down_sync(0xffffffffu, r1, o);
          const float z0 = __shfl_up_sync(0xffffffffu, w0, o);
          const float z1 = __shfl_up_sync(0xffffffffu, w1, o);
          if (lane + o < 32) {
            r0 += y0;
            r1 += y1;
          }
          if (lane >= o) {
            w0 += z0;
            w1 += z1;
          }
        }
        const float r1all = __shfl_sync(0xffffffffu, r1, 0);
        const float w0all = __shfl_sync(0xffffffffu, w0, 31);
        const float from = warp == 1 ? r0 + r1all : r1;
        // (what t writes may be large, and is not part of it)
        float before = __shfl_up_sync(0xffffffffu, warp == 1 ? w0 : w1, 1);
        if (lane == 0) before = 0.f;
        if (warp == 2) before += w0all;
        if (t < rows) {
          const int64_t at = ((int64_t)b * a.L + (int64_t)c * kC + t) * a.H + h;
          a.dbeta[at] = (warp == 1 ? p0 : p1) + s.total[t];
          // (a state that starts anew at t leaves t nothing to decay: all four are 0)
          a.dg[at] = vec[kVecs * kC] * total + from + before + near;
        }
      }
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMmaWarp) {
    tc::tmem_relinquish();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int KP>
cudaError_t run(const Args& a, cudaStream_t st) {
  CUtensorMap mq, mk, md, moq, mok;
  const TokStride dense = {a.L * a.G * a.K, (int64_t)a.G * a.K};
  if (!token_map(&mq, a.q, a.qcols, a.G, a.L, a.B, a.sq, true) ||
      !token_map(&mk, a.k, a.kcols, a.G, a.L, a.B, a.sk, true) ||
      !token_map(&md, a.dout, a.docols, a.H, a.L, a.B, a.sdo, true))
    return cudaErrorInvalidValue;
  const int tma_out = !a.dq_part && a.K % 8 == 0 && (((uintptr_t)a.dq | (uintptr_t)a.dk) & 15) == 0;
  moq = mok = mq;
  if (tma_out && (!token_map(&moq, a.dq, a.K, a.G, a.L, a.B, dense, true) ||
                  !token_map(&mok, a.dk, a.K, a.G, a.L, a.B, dense, true)))
    return cudaErrorInvalidValue;
  const int smem = (int)sizeof(Smem<KP>) + 1024;
  const cudaError_t e = cudaFuncSetAttribute(
      tc_grads_kernel<KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t chunks = (int64_t)a.B * a.H * a.nc;
  const int grid = (int)(chunks < row::sm_count() ? chunks : row::sm_count());
  g_launched = true;
  tc_grads_kernel<KP><<<grid, kThreads, smem, st>>>(mq, mk, md, moq, mok, tma_out, a);
  return cudaGetLastError();
}
static_assert(sizeof(Smem<128>) + 1024 <= 227 * 1024, "shared memory");

}  // namespace grd

int tc_grads_status(int reset, cudaStream_t st, int* bits) {
  return read_status(grd::g_status, grd::g_launched, reset, st, bits);
}
cudaError_t launch_tc_grads(const Args& a, cudaStream_t st) {
  const cudaError_t e = a.KP == 64 ? grd::run<64>(a, st) : grd::run<128>(a, st);
  return e != cudaSuccess || !a.dq_part ? e : launch_group_sum<bf16>(a, st);
}

}  // namespace delta
}  // namespace ssd
