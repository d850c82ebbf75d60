// The gated delta rule's forward in bf16 on tcgen05, one CTA per SM, each at one
// segment of a (batch row, head, 128 channels), chunk after chunk.
//
// Transposed as in ssd_delta_fwd.cu: TMEM lane = channel, columns = tokens or
// dstate.  Per chunk, with S in the registers of sixteen warps (a row and a quarter
// of dstate a thread) and as two bf16 terms in TMEM:
//   Y = S K^T, then O1 = S Q^T           A: S
//   y = v - e^G Y  -> TMEM               the chain's warps
//   X = y T^T                            A: y, over Y's columns
//   w = beta e^(G_C - G) X -> TMEM
//   W = w K, then O2 = X P^T             A: w in S's columns; x over X's columns
//   S = e^(G_C) S + W -> TMEM
// and beside it out = scale e^G O1 + O2 (P holds scale and beta).  K^T and K are
// one tile read in both orders.  Roles, so that only the chain Y - y - X - w - W - S
// is in a chunk's way:
//   warps 0-15   the chain, a quarter of the lanes and of the columns each (its
//                phases are bound by their warps' latency: half as many columns a
//                warp take about half as long)
//   warps 16-19  out
//   warp 20      issues the MMAs;  21: the copies
// Shared and tensor memory: one CTA an SM.
// Bound by that chain: of a chunk's 5200 to 5900 cycles its MMAs take 1750 (Y 704, X
// 528, W 512) and their commits 600, the three steps between them 600 to 1000 each.
// 8 x 4096 tokens of 40 heads (20480 chunks): 463 us (480 with Y and O1 in one product,
// which is the shorter of the two, but all of it in the chain's way).  With S0 and X kept
// for a backward 4 x 4096 tokens take 400 us: 192 KB a chunk and head, 4.9 TB/s.
#include "ssd_delta_tc.cuh"

namespace ssd {
namespace delta {
namespace fwd {

constexpr int kChainWarps = 16, kOutWarp = 16, kMmaWarp = 20, kLoadWarp = 21;
constexpr int kThreads = 24 * 32;   // (warps 22 and 23 fill the last warpgroup)
// Registers a thread: launched with 80, six warps a quadrant of the SM:
// 4 x 80 + 104 + 48 = 472 of 480
constexpr int kTP = 2;   // stages
// TMEM columns: S's terms (and w's), Y / y, O1, X / x, O2, W
constexpr uint32_t kAS = 0, kR0 = 128, kO1 = 192, kR1 = 256, kO2 = 320, kW = 384;

template <int KP, bool KEEP>
struct Smem {
  static constexpr int kKQ = KEEP ? 2 : 3;
  static constexpr uint32_t kHalf = 2 * kTile;   // 64 columns: 64 rows of K, 64 of Q
  unsigned char kq[kKQ][KP / 64][2][kTile];
  unsigned char v[2][2][kTile];                  // [channel half][token][64], not swizzled
  unsigned char o[2][kTile];                     // out, as v
  unsigned char x[KEEP ? 2 : 0][2][kTile];       // x's terms: [term][channel half][token][64]
  unsigned char tp[kTP][4][kTile];               // T's terms, P's terms
  alignas(16) float vec[kTP][vec_floats<kC>()];
  uint64_t kq_full[kKQ], kq_empty[kKQ], v_full[2], v_empty[2], tp_full[kTP], tp_empty[kTP],
      vec_full[kTP], vec_empty[kTP];
  uint64_t s_ready, y_done, yt_ready, x_done, w_ready, w_done, o_done, o1_read, o2_read,
      o_sync, slot_done, mma_drain;
  Items items;
  uint32_t tmem;
  volatile int gave_up;
};

__device__ int g_status;
std::atomic<bool> g_launched{false};

template <int KP, bool KEEP>
__global__ void __launch_bounds__(kThreads, 1)
    tc_forward_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo,
                      const __grid_constant__ Args a) {
  extern __shared__ unsigned char raw[];
  using S = Smem<KP, KEEP>;
  constexpr int kKQ = S::kKQ;
  S& s = *reinterpret_cast<S*>(raw + ((1024 - (saddr(raw) & 1023)) & 1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nc = a.nc;
  if (warp == kMmaWarp) tc::tmem_alloc(&s.tmem, 512);
  if (tid == 0) {
    for (int i = 0; i < kKQ; ++i) {
      tc::mbar_init(&s.kq_full[i], 1);
      tc::mbar_init(&s.kq_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s.v_full[i], 1);
      tc::mbar_init(&s.v_empty[i], kChainWarps);
      tc::mbar_init(&s.tp_full[i], 1);
      tc::mbar_init(&s.tp_empty[i], 1);
      tc::mbar_init(&s.vec_full[i], 1);
      tc::mbar_init(&s.vec_empty[i], kChainWarps + 4);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s.items.full[i], 1);
      tc::mbar_init(&s.items.empty[i], kChainWarps + 5);   // ... out's four, the MMAs' one
    }
    tc::mbar_init(&s.s_ready, kChainWarps);
    tc::mbar_init(&s.yt_ready, kChainWarps);
    tc::mbar_init(&s.w_ready, kChainWarps);
    tc::mbar_init(&s.o1_read, 4);
    tc::mbar_init(&s.o2_read, 4);
    tc::mbar_init(&s.o_sync, 4);
    tc::mbar_init(&s.slot_done, kChainWarps);
    tc::mbar_init(&s.y_done, 1);
    tc::mbar_init(&s.x_done, 1);
    tc::mbar_init(&s.w_done, 1);
    tc::mbar_init(&s.o_done, 1);
    tc::mbar_init(&s.mma_drain, 1);
    tc::mbar_fence_init();
    s.gave_up = 0;
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s.tmem;
  auto W = [&](uint64_t* bar, uint32_t parity) { wait_for(bar, parity, &s.gave_up, &g_status); };
  // the CTA's n-th item, for all lanes of a warp (bh < 0: no more)
  auto item = [&](int n) {
    W(&s.items.full[n & 1], (n >> 1) & 1);
    Item i = s.items.item[n & 1];
    warp_arrive(&s.items.empty[n & 1], lane);
    if (__any_sync(0xffffffffu, s.gave_up)) i.bh = -1;
    return i;
  };

  if (warp >= kMmaWarp) {
    SSD_SETREG("dec", "48");
    if (warp == kLoadWarp) {
      int n = 0;   // chunks so far
      bool go = true;
      for (int k = 0; go; ++k) {
        int ticket = 0;
        if (lane == 0) ticket = atomicAdd(a.ctrl, 1);
        const Item it = item_of(a, __shfl_sync(0xffffffffu, ticket, 0));
        if (k >= 2) W(&s.items.empty[k & 1], (k / 2 - 1) & 1);
        if (lane == 0) s.items.item[k & 1] = it;
        warp_arrive(&s.items.full[k & 1], lane);
        if (it.bh < 0) break;
        const int b = it.bh / a.H, h = it.bh % a.H, kg = h / (a.H / a.G);
        for (int c = it.first; c < it.last; ++c, ++n) {
          const int p = n & 1, kq = n % kKQ;
          const uint32_t ph = (n / 2 - 1) & 1;
          const int64_t id = (int64_t)it.bh * nc + c;
          if (n >= kKQ) W(&s.kq_empty[kq], (n / kKQ - 1) & 1);
          if (__any_sync(0xffffffffu, s.gave_up)) {
            go = false;
            break;
          }
          if (tc::elect_one()) {
            tc::mbar_arrive_expect_tx(&s.kq_full[kq], KP / 64 * 2 * kTile);
            for (int i = 0; i < KP / 64; ++i) {
              tc::tma_load_4d(s.kq[kq][i][0], &mk, &s.kq_full[kq], i * 64, kg, c * kC, b);
              tc::tma_load_4d(s.kq[kq][i][1], &mq, &s.kq_full[kq], i * 64, kg, c * kC, b);
            }
          }
          __syncwarp();
          // (after a wait that gave up, what follows is only waited for)
          if (n >= 2) W(&s.v_empty[p], ph);
          if (tc::elect_one()) {
            tc::mbar_arrive_expect_tx(&s.v_full[p], 2 * kTile);
            for (int i = 0; i < 2; ++i)
              tc::tma_load_4d(s.v[p][i], &mv, &s.v_full[p], it.v0 + i * 64, h, c * kC, b);
          }
          __syncwarp();
          if (n >= 2) W(&s.vec_empty[p], ph);
          if (n >= 2) W(&s.tp_empty[p], ph);
          if (tc::elect_one()) {
            tc::mbar_arrive_expect_tx(&s.vec_full[p], vec_floats<kC>() * 4);
            tc::bulk_load(s.vec[p], a.vec + id * vec_floats<kC>(), vec_floats<kC>() * 4,
                          &s.vec_full[p]);
            tc::mbar_arrive_expect_tx(&s.tp_full[p], 4 * kTile);
            tc::bulk_load(s.tp[p], reinterpret_cast<const unsigned char*>(a.T) + id * 4 * kTile,
                          4 * kTile, &s.tp_full[p]);
          }
          __syncwarp();
        }
      }
      // every copy has landed before the CTA ends
      for (int i = n > kKQ ? n - kKQ : 0; i < n; ++i) {
        drain(&s.kq_full[i % kKQ], (i / kKQ) & 1, &g_status);
        if (i < n - 2) continue;
        drain(&s.tp_full[i & 1], (i / 2) & 1, &g_status);
        drain(&s.vec_full[i & 1], (i / 2) & 1, &g_status);
        drain(&s.v_full[i & 1], (i / 2) & 1, &g_status);
      }
    } else if (warp == kMmaWarp) {
      // (the warp stays converged, one elected lane issuing: descriptors then live
      // in uniform registers)
      constexpr uint32_t id64 = tc::idesc_bf16(128, 64, false, false);
      constexpr uint32_t idw = tc::idesc_bf16(128, KP, false, true);
      constexpr uint32_t half = S::kHalf >> 4;
      constexpr uint32_t lo = kTile >> 4;   // a tile's second term
      const uint64_t dk0 = tc::sdesc_sw128(saddr(s.kq[0][0][0]), 16, 1024);
      const uint64_t dm0 = tc::sdesc_sw128(saddr(s.kq[0][0][0]), S::kHalf, 1024);
      const uint64_t dt0 = tc::sdesc_sw128(saddr(s.tp[0][0]), 16, 1024);
      const uint64_t dp0 = tc::sdesc_sw128(saddr(s.tp[0][2]), 16, 1024);
      auto stop = [&] { return __any_sync(0xffffffffu, s.gave_up) != 0; };
      int st = 0;
      uint32_t kq_ph = 0;
      int n = 0, end = 0;
      for (int k = 0;; ++n) {
        if (n == end) {
          const Item it = item(k++);
          if (it.bh < 0) break;
          end = n + it.last - it.first;
        }
        const uint32_t ph = n & 1, tp = n & 1;
        const uint32_t fill = (n >> 1) & 1;
        const uint64_t dk = dk0 + st * ((KP / 64) * S::kHalf >> 4);
        const uint64_t dm = dm0 + st * ((KP / 64) * S::kHalf >> 4);
        const uint64_t dt = dt0 + tp * (4 * kTile >> 4), dp = dp0 + tp * (4 * kTile >> 4);
        W(&s.kq_full[st], kq_ph);
        W(&s.s_ready, ph);
        if (stop()) break;
        tc::fence_after_sync();
        if (tc::elect_one()) {
          mma_chain<KP / 16, false>(tmem + kR0, tmem + kAS, 1, dk, half, id64, true);
          mma_chain<KP / 16, false>(tmem + kR0, tmem + kAS, 0, dk, half, id64, false);
          tc::mma_commit(&s.y_done);
        }
        __syncwarp();
        if (n > 0) W(&s.o1_read, ph ^ 1);
        if (stop()) break;
        tc::fence_after_sync();
        if (tc::elect_one()) {   // (while the chain's warps are at y)
          mma_chain<KP / 16, false>(tmem + kO1, tmem + kAS, 1, dk + lo, half, id64, true);
          mma_chain<KP / 16, false>(tmem + kO1, tmem + kAS, 0, dk + lo, half, id64, false);
        }
        __syncwarp();
        W(&s.tp_full[tp], fill);
        if (n > 0) W(&s.o2_read, ph ^ 1);   // O2 and x's terms of the chunk before
        W(&s.yt_ready, ph);
        if (stop()) break;
        tc::fence_after_sync();
        if (tc::elect_one()) {
          mma_chain<4, false>(tmem + kR1, tmem + kR0, 1, dt, 0, id64, true);
          mma_chain<4, false>(tmem + kR1, tmem + kR0, 0, dt + lo, 0, id64, false);
          mma_chain<4, false>(tmem + kR1, tmem + kR0, 0, dt, 0, id64, false);
          tc::mma_commit(&s.x_done);
        }
        __syncwarp();
        W(&s.w_ready, ph);
        if (stop()) break;
        tc::fence_after_sync();
        if (tc::elect_one()) {
          mma_chain<4, true>(tmem + kW, tmem + kAS, 1, dm, 0, idw, true);
          mma_chain<4, true>(tmem + kW, tmem + kAS, 0, dm, 0, idw, false);
          tc::mma_commit(&s.w_done);
          tc::mma_commit(&s.kq_empty[st]);
          mma_chain<4, false>(tmem + kO2, tmem + kR1, 1, dp, 0, id64, true);
          mma_chain<4, false>(tmem + kO2, tmem + kR1, 0, dp + lo, 0, id64, false);
          mma_chain<4, false>(tmem + kO2, tmem + kR1, 0, dp, 0, id64, false);
          tc::mma_commit(&s.o_done);
          tc::mma_commit(&s.tp_empty[tp]);
        }
        __syncwarp();
        if (++st == kKQ) {
          st = 0;
          kq_ph ^= 1;
        }
      }
      if (tc::elect_one()) tc::mma_commit(&s.mma_drain);
      __syncwarp();
      drain(&s.mma_drain, 0, &g_status);
    }
  } else if (warp >= kOutWarp) {
    // ---------------- out = scale e^G O1 + O2
    SSD_SETREG("inc", "104");
    const int qr = warp & 3, row = qr * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)qr << 21);
    // (the four warps; a wait that gives up, unlike a barrier, lets every warp end)
    auto together = [&](uint32_t phase) {
      warp_arrive(&s.o_sync, lane);
      W(&s.o_sync, phase);
    };
    Item it = {};
    int c = 0;
    for (int n = 0, k = 0;; ++n, ++c) {
      if (c == it.last) {
        it = item(k++);
        if (it.bh < 0) break;
        c = it.first;
      }
      const int b = it.bh / a.H, h = it.bh % a.H, v0 = it.v0, vr = v0 + row;
      const uint32_t ph = n & 1;
      const float* gam = s.vec[ph] + kGam * kC;
      unsigned char* const vt = s.o[row >> 6] + (row & 63) * 2;
      float x[4][16];
      W(&s.x_done, ph);   // O1 is done as X is
      tc::fence_after_sync();
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        uint32_t r[16];
        tc::tmem_ld16(lanes + kO1 + p * 16, r);
        tc::tmem_ld_wait_regs(r);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[p][i] = __uint_as_float(r[i]) * a.scale;
      }
      tc::fence_before_sync();
      warp_arrive(&s.o1_read, lane);
#pragma unroll
      for (int p = 0; p < 4; ++p) scale_by(x[p], gam + p * 16);
      if (warp == kOutWarp && tc::elect_one()) tc::bulk_wait_read();   // the tiles' last copies
      together(0);
      W(&s.o_done, ph);
      tc::fence_after_sync();
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        uint32_t r[16];
        tc::tmem_ld16(lanes + kO2 + p * 16, r);
        tc::tmem_ld_wait_regs(r);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[p][i] += __uint_as_float(r[i]);
        if (KEEP) {
          tc::tmem_ld16(lanes + kR1 + p * 16, r);
          tc::tmem_ld_wait_regs(r);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            unsigned char* at =
                s.x[0][row >> 6] + tile_at<64>(p * 16 + i, (row & 63) >> 3) + (row & 7) * 2;
            const int sh = 16 * (i & 1);
            *reinterpret_cast<uint16_t*>(at) = (uint16_t)(r[i >> 1] >> sh);
            *reinterpret_cast<uint16_t*>(at + 2 * kTile) = (uint16_t)(r[8 + (i >> 1)] >> sh);
          }
        }
      }
      tc::fence_before_sync();
      warp_arrive(&s.o2_read, lane);
      warp_arrive(&s.vec_empty[ph], lane);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        if (a.wide_out) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            *reinterpret_cast<bf16*>(vt + (p * 16 + i) * 128) = __float2bfloat16_rn(x[p][i]);
        } else if (a.out && vr < a.V && a.pass != kParts) {   // rows off 16 bytes
          const int64_t t0 = (int64_t)c * kC + p * 16;
          bf16* dst = static_cast<bf16*>(a.out) + (((int64_t)b * a.L + t0) * a.H + h) * a.V + vr;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (t0 + i < a.L) dst[(int64_t)i * a.H * a.V] = __float2bfloat16_rn(x[p][i]);
        }
      }
      tc::fence_proxy_async_smem();
      together(1);
      if (warp == kOutWarp) {
        if (tc::elect_one()) {
          if (a.wide_out && !s.gave_up && a.pass != kParts)
            for (int i = 0; i < 2; ++i)
              if (v0 + i * 64 < a.V) tc::tma_store_4d(&mo, s.o[i], v0 + i * 64, h, c * kC, b);
          if (KEEP && !s.gave_up) {
            // planes [term][channel half][token][64] of the workspace
            unsigned char* to = reinterpret_cast<unsigned char*>(a.X) +
                                (((int64_t)it.bh * nc + c) * 2 * (a.VP / 64) + v0 / 64) * kTile;
            for (int i = 0; i < 2; ++i)
              asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                               to + (int64_t)i * (a.VP / 64) * kTile),
                           "r"(saddr(s.x[i][0])), "r"(2 * kTile)
                           : "memory");
          }
          tc::bulk_commit();
        }
        __syncwarp();
      }
    }
    if (warp == kOutWarp && tc::elect_one()) tc::bulk_wait_all();
  } else {
    // ---------------- the chain
    const int qr = warp & 3, part = warp >> 2, row = qr * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)qr << 21);   // this warp's 32 TMEM lanes
    constexpr int SP = KP / 64;                           // pieces of 16 of S a thread
    float S0[SP][16];
    Item it = {};
    // A piece of S as terms to TMEM (and to memory, as chunk c's first state)
    auto put_state = [&](int p, int c) {
      uint32_t t[16];
      two_terms(S0[p], t);
      tc::tmem_st16(lanes + kAS + (part * SP + p) * 16, t);
      if (KEEP) keep_row<KP>(t, a.S0, (int64_t)it.bh * nc + c, it.v0 + row, (part * SP + p) * 16, a);
    };
    auto told = [&](uint64_t* bar) {   // what this warp wrote to TMEM is there
      tc::tmem_st_wait();
      tc::fence_before_sync();
      warp_arrive(bar, lane);
    };
    int c = 0, slots = 0;
    for (int n = 0, k = 0;; ++n, ++c) {
      if (c == it.last) {
        it = item(k++);
        if (it.bh < 0) break;
        c = it.first;
        if (c == 0) {
          read_row<SP>(S0, a.init, it.bh, it.v0 + row, part, a);
        } else if (a.pass == kParts) {
#pragma unroll
          for (int p = 0; p < SP; ++p)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              S0[p][i] = it.unit && row == (part * SP + p) * 16 + i ? 1.f : 0.f;
        } else {
          if (lane == 0 && a.pass == kWhole)
            wait_flag(flag_of(a, it), c / a.seg, &s.gave_up, &g_status);
          __syncwarp();
          read_slot<SP>(S0, a, it, row, part);
        }
#pragma unroll
        for (int p = 0; p < SP; ++p) put_state(p, c);
        told(&s.s_ready);
      }
      const uint32_t ph = n & 1;
      const float* vec = s.vec[ph];
      const unsigned char* const vt = s.v[ph][row >> 6] + (row & 63) * 2;
      uint32_t r[16], t[16];
      float x[16];
      const int t0 = part * 16;   // the warp's tokens
      // y = v - e^G Y
      W(&s.v_full[ph], (n >> 1) & 1);
      W(&s.vec_full[ph], (n >> 1) & 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {   // v's pairs of tokens, while Y is computed
        const unsigned char* q = vt + (t0 + 2 * i) * 128;
        t[i] = it.unit ? 0u
                       : *reinterpret_cast<const uint16_t*>(q) |
                             (uint32_t)*reinterpret_cast<const uint16_t*>(q + 128) << 16;
      }
      W(&s.y_done, ph);
      tc::fence_after_sync();
      tc::tmem_ld16(lanes + kR0 + t0, r);
      tc::tmem_ld_wait_regs(r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 f = *reinterpret_cast<const float4*>(vec + kRead * kC + t0 + 4 * i);
        fma2(x[4 * i], x[4 * i + 1], __uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]), f.x,
             f.y, lo_of(t[2 * i]), hi_of(t[2 * i]));
        fma2(x[4 * i + 2], x[4 * i + 3], __uint_as_float(r[4 * i + 2]),
             __uint_as_float(r[4 * i + 3]), f.z, f.w, lo_of(t[2 * i + 1]), hi_of(t[2 * i + 1]));
      }
      two_terms(x, r);
      tc::tmem_st16(lanes + kR0 + t0, r);
      told(&s.yt_ready);
      warp_arrive(&s.v_empty[ph], lane);
      // x's terms, and w = beta e^(G_C - G) x
      W(&s.x_done, ph);
      tc::fence_after_sync();
      tc::tmem_ld16(lanes + kR1 + t0, r);
      tc::tmem_ld_wait_regs(r);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
      two_terms(x, t);
      tc::tmem_st16(lanes + kR1 + t0, t);
      scale_by(x, vec + kWrite * kC + t0);
      two_terms(x, r);
      tc::tmem_st16(lanes + kAS + t0, r);
      told(&s.w_ready);
      const float through = vec[kVecs * kC];
      warp_arrive(&s.vec_empty[ph], lane);
      // S = e^(G_C) S + W
      W(&s.w_done, ph);
      tc::fence_after_sync();
#pragma unroll
      for (int p = 0; p < SP; ++p) {
        tc::tmem_ld16(lanes + kW + (part * SP + p) * 16, r);
        tc::tmem_ld_wait_regs(r);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          fma2(S0[p][2 * i], S0[p][2 * i + 1], S0[p][2 * i], S0[p][2 * i + 1], through, through,
               __uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
        if (c + 1 < it.last) put_state(p, c + 1);
      }
      if (c + 1 < it.last) {
        told(&s.s_ready);
      } else if (a.pass == kParts) {
        write_slot<SP>(S0, a, it, row, part);
      } else if (c + 1 < nc) {   // on to the next segment
        if (a.pass == kJoined) continue;
        write_slot<SP>(S0, a, it, row, part);
        warp_arrive(&s.slot_done, lane);
        if (warp == 0) {
          W(&s.slot_done, slots++ & 1);
          if (lane == 0) raise_flag(flag_of(a, it), (c + 1) / a.seg);
        }
      } else {
        write_row<SP>(S0, a.final, it.bh, it.v0 + row, part, a);
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

template <int KP, bool KEEP>
cudaError_t run(const Args& a, cudaStream_t st) {
  CUtensorMap mq, mk, mv, mo;
  const TokStride dense = {a.L * a.H * a.V, (int64_t)a.H * a.V};
  if (!token_map(&mq, a.q, a.qcols, a.G, a.L, a.B, a.sq, true) ||
      !token_map(&mk, a.k, a.kcols, a.G, a.L, a.B, a.sk, true) ||
      !token_map(&mv, a.v, a.vcols, a.H, a.L, a.B, a.sv, false))
    return cudaErrorInvalidValue;
  mo = mv;
  if (a.wide_out && !token_map(&mo, a.out, a.V, a.H, a.L, a.B, dense, false))
    return cudaErrorInvalidValue;
  const int smem = (int)sizeof(Smem<KP, KEEP>) + 1024;
  cudaError_t e = cudaFuncSetAttribute(
      tc_forward_kernel<KP, KEEP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  int grid = 0;
  e = start_work(a, &grid, st);
  if (e != cudaSuccess) return e;
  g_launched = true;
  tc_forward_kernel<KP, KEEP><<<grid, kThreads, smem, st>>>(mq, mk, mv, mo, a);
  return cudaGetLastError();
}
static_assert(sizeof(Smem<128, false>) + 1024 <= 227 * 1024 &&
              sizeof(Smem<128, true>) + 1024 <= 227 * 1024, "shared memory");

}  // namespace fwd

// Status bits of the launches that gave up a wait (host; ssd_scan_status).
int tc_forward_status(int reset, cudaStream_t st, int* bits) {
  return read_status(fwd::g_status, fwd::g_launched, reset, st, bits);
}

// S <- S M + W from segment to segment, eight rows a CTA, in fp32: a thread has four
// columns of a row; S's rows and M stand in shared memory, the next M on its way (rows
// padded, or every fourth lane would meet in a bank).  A segment is a product of 8 x
// 128 x 128 behind the one before it: five of them for 16 heads take 24 us.
template <int KP>
__global__ void __launch_bounds__(KP * 2) tc_join_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) unsigned char raw[];
  // rows a bank group apart: M [2][KP / 4][KP], S [2][8][KP]
  constexpr int PM = KP + 1, PS = KP + 4;
  float4* const m = reinterpret_cast<float4*>(raw);
  float* const s = reinterpret_cast<float*>(m + 2 * (KP / 4) * PM);
  const int vb = (a.V + 127) / 128, n = a.B * a.H * vb, tid = threadIdx.x;
  const int lane = blockIdx.x, r = tid & 7, row = blockIdx.y * 8 + r, col = tid >> 3;
  float4* const slots = reinterpret_cast<float4*>(a.slots);
  const int64_t size = 32 * KP;   // of a slot, in float4
  auto load = [&](int seg) {
    const float4* src =
        slots + ((int64_t)n * (a.segs - 1) + (int64_t)(seg - 1) * a.B * a.H + lane / vb) * size;
    float4* dst = m + (seg & 1) * (KP / 4) * PM;
    for (int i = tid; i < KP / 4 * KP; i += KP * 2)   // rows below KP of 128
      cp16(saddr(dst + i / KP * PM + i % KP), src + i / KP * 128 + i % KP, 16);
    cp_commit();
  };
  if (a.segs > 2) load(1);
  float4 x = slots[(int64_t)lane * size + col * 128 + row];
  for (int seg = 1; seg + 1 < a.segs; ++seg) {
    float* const now = s + (seg & 1) * 8 * PS;
    *reinterpret_cast<float4*>(now + r * PS + col * 4) = x;
    float4* const w = slots + ((int64_t)seg * n + lane) * size + col * 128 + row;
    x = *w;
    if (seg + 2 < a.segs) load(seg + 1);
    else cp_commit();
    cp_wait<1>();
    __syncthreads();
    const float4* const f = m + ((seg & 1) * (KP / 4) + col) * PM;
#pragma unroll 4
    for (int k = 0; k < KP; k += 4) {
      const float4 y4 = *reinterpret_cast<const float4*>(now + r * PS + k);
      const float y[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 g = f[k + e];
        x.x = fmaf(y[e], g.x, x.x);
        x.y = fmaf(y[e], g.y, x.y);
        x.z = fmaf(y[e], g.z, x.z);
        x.w = fmaf(y[e], g.w, x.w);
      }
    }
    *w = x;
    __syncthreads();   // this M's place is the one after the next's
  }
  cp_wait<0>();
}

template <int KP>
cudaError_t join(const Args& a, cudaStream_t st) {
  const int smem = 2 * (KP / 4) * (KP + 1) * 16 + 2 * 8 * (KP + 4) * 4;
  const cudaError_t e =
      cudaFuncSetAttribute(tc_join_kernel<KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(a.B * a.H * ((a.V + 127) / 128)), 16);
  tc_join_kernel<KP><<<grid, KP * 2, smem, st>>>(a);
  return cudaGetLastError();
}
cudaError_t launch_tc_join(const Args& a, cudaStream_t st) {
  return a.KP == 64 ? join<64>(a, st) : join<128>(a, st);
}

cudaError_t launch_tc_forward(const Args& args, cudaStream_t st) {
  Args a = args;
  if (a.pass == kParts) {
    Args f = a;
    f.S0 = f.X = nullptr;
    f.final = nullptr;
    cudaError_t e = a.KP == 64 ? fwd::run<64, false>(f, st) : fwd::run<128, false>(f, st);
    if (e == cudaSuccess) e = launch_tc_join(f, st);
    if (e == cudaSuccess) e = copy_first(a, &a.init, a.final, st);
    if (e != cudaSuccess) return e;
    a.pass = kJoined;
  }
  if (a.KP == 64) return a.S0 ? fwd::run<64, true>(a, st) : fwd::run<64, false>(a, st);
  return a.S0 ? fwd::run<128, true>(a, st) : fwd::run<128, false>(a, st);
}

}  // namespace delta
}  // namespace ssd
