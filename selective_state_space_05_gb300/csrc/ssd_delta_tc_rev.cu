// The gated delta rule's backward along the sequence on tcgen05, last chunk first:
// one CTA per SM, which takes (segment, head, 128 channels) items by tickets as the
// forward's do, transposed as there, with the state's gradient dS in registers and as two
// bf16 terms in TMEM.
// Per chunk:
//   Z = dS K^T                                A: dS
//   dx = beta e^(G_C - G) Z + do P -> TMEM     (do P ahead: A: do, one term)
//   dY = dx T                                 A: dx, over Z's columns
//   -e^G dY -> TMEM                           dY is the gradient of v
//   W = (scale e^G do) Q + (-e^G dY) K        (the first ahead)
//   dS = e^(G_C) dS + W -> TMEM
// P and T are read with tokens along K here, the same tiles as the forward's.
// Roles: warps 0-15 the chain, 16-19 do into TMEM for the next chunk and dY out of
// it, 20 issues the MMAs, 21 the copies.  dS after each chunk and dY are kept as
// terms for the chunks' own gradients.
// Bound by the chain dS - Z - dx - dY - W - dS as the forward, and by HBM: 10240 chunks of
// 4 x 4096 tokens and 40 heads in 406 us, 4.9 TB/s (96 KB of 192 a chunk are kept).
#include "ssd_delta_tc.cuh"

namespace ssd {
namespace delta {
namespace rev {

constexpr int kChainWarps = 16, kIoWarp = 16, kMmaWarp = 20, kLoadWarp = 21;
constexpr int kThreads = 24 * 32;   // (warps 22 and 23 fill the last warpgroup)
// Registers a thread: as the forward's, 4 x 80 + 104 + 48 of 480 a quadrant
// TMEM columns: dS's terms (and dY's), Z / dx, do P / dY, W, scale e^G do, do
constexpr uint32_t kAS = 0, kZ = 128, kY = 192, kW = 256, kA1 = 384, kAD = 448;

template <int KP>
struct Smem {
  static constexpr uint32_t kHalf = 2 * kTile;   // 64 columns: 64 rows of K, 64 of Q
  unsigned char kq[2][KP / 64][2][kTile];
  unsigned char d[2][2][kTile];                  // dout: [channel half][token][64], not swizzled
  unsigned char y[2][2][kTile];                  // dY's terms: [term][channel half][token][64]
  unsigned char tp[2][4][kTile];                 // T's terms, P's terms
  alignas(16) float vec[2][vec_floats<kC>()];
  uint64_t kq_full[2], kq_empty[2], d_full[2], d_empty[2], tp_full[2], tp_empty[2], vec_full[2],
      vec_empty[2];
  uint64_t s_ready, z_done, xt_ready, y_done, w_ready, w_done, in_ready, io_sync, slot_done,
      mma_drain;
  Items items;
  uint32_t tmem;
  volatile int gave_up;
};

__device__ int g_status;
std::atomic<bool> g_launched{false};

template <int KP>
__global__ void __launch_bounds__(kThreads, 1)
    tc_reverse_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap md, const __grid_constant__ CUtensorMap mv,
                      const __grid_constant__ Args a) {
  extern __shared__ unsigned char raw[];
  using S = Smem<KP>;
  S& s = *reinterpret_cast<S*>(raw + ((1024 - (saddr(raw) & 1023)) & 1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nc = a.nc;
  if (warp == kMmaWarp) tc::tmem_alloc(&s.tmem, 512);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s.kq_full[i], 1);
      tc::mbar_init(&s.kq_empty[i], 1);
      tc::mbar_init(&s.d_full[i], 1);
      tc::mbar_init(&s.d_empty[i], 4);
      tc::mbar_init(&s.tp_full[i], 1);
      tc::mbar_init(&s.tp_empty[i], 1);
      tc::mbar_init(&s.vec_full[i], 1);
      tc::mbar_init(&s.vec_empty[i], kChainWarps + 4);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s.items.full[i], 1);
      tc::mbar_init(&s.items.empty[i], kChainWarps + 5);   // ... io's four, the MMAs' one
    }
    tc::mbar_init(&s.s_ready, kChainWarps);
    tc::mbar_init(&s.xt_ready, kChainWarps);
    tc::mbar_init(&s.w_ready, kChainWarps);
    tc::mbar_init(&s.in_ready, 4);
    tc::mbar_init(&s.io_sync, 4);
    tc::mbar_init(&s.slot_done, kChainWarps);
    tc::mbar_init(&s.z_done, 1);
    tc::mbar_init(&s.y_done, 1);
    tc::mbar_init(&s.w_done, 1);
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
  // the CTA's n-th item, for all lanes of a warp (bh < 0: no more); its chunks count
  // from the sequence's end
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
        for (int r = it.first; r < it.last; ++r, ++n) {
          const int c = nc - 1 - r, p = n & 1;
          const uint32_t ph = (n / 2 - 1) & 1;
          const int64_t id = (int64_t)it.bh * nc + c;
          if (n >= 2) W(&s.d_empty[p], ph);
          if (n >= 2) W(&s.vec_empty[p], ph);
          if (__any_sync(0xffffffffu, s.gave_up)) {
            go = false;
            break;
          }
          if (tc::elect_one()) {
            tc::mbar_arrive_expect_tx(&s.d_full[p], 2 * kTile);
            for (int i = 0; i < 2; ++i)
              tc::tma_load_4d(s.d[p][i], &md, &s.d_full[p], it.v0 + i * 64, h, c * kC, b);
            tc::mbar_arrive_expect_tx(&s.vec_full[p], vec_floats<kC>() * 4);
            tc::bulk_load(s.vec[p], a.vec + id * vec_floats<kC>(), vec_floats<kC>() * 4,
                          &s.vec_full[p]);
          }
          __syncwarp();
          // (after a wait that gave up, what follows is only waited for)
          if (n >= 2) W(&s.tp_empty[p], ph);
          if (n >= 2) W(&s.kq_empty[p], ph);
          if (tc::elect_one()) {
            tc::mbar_arrive_expect_tx(&s.tp_full[p], 4 * kTile);
            tc::bulk_load(s.tp[p], reinterpret_cast<const unsigned char*>(a.T) + id * 4 * kTile,
                          4 * kTile, &s.tp_full[p]);
            tc::mbar_arrive_expect_tx(&s.kq_full[p], KP / 64 * 2 * kTile);
            for (int i = 0; i < KP / 64; ++i) {
              tc::tma_load_4d(s.kq[p][i][0], &mk, &s.kq_full[p], i * 64, kg, c * kC, b);
              tc::tma_load_4d(s.kq[p][i][1], &mq, &s.kq_full[p], i * 64, kg, c * kC, b);
            }
          }
          __syncwarp();
        }
      }
      // every copy has landed before the CTA ends
      for (int i = n > 2 ? n - 2 : 0; i < n; ++i) {
        drain(&s.kq_full[i & 1], (i / 2) & 1, &g_status);
        drain(&s.tp_full[i & 1], (i / 2) & 1, &g_status);
        drain(&s.vec_full[i & 1], (i / 2) & 1, &g_status);
        drain(&s.d_full[i & 1], (i / 2) & 1, &g_status);
      }
    } else if (warp == kMmaWarp) {
      constexpr uint32_t id64 = tc::idesc_bf16(128, 64, false, false);
      constexpr uint32_t id64m = tc::idesc_bf16(128, 64, false, true);
      constexpr uint32_t idw = tc::idesc_bf16(128, KP, false, true);
      constexpr uint32_t half = S::kHalf >> 4;
      constexpr uint32_t lo = kTile >> 4;   // a tile's second term
      const uint64_t dk0 = tc::sdesc_sw128(saddr(s.kq[0][0][0]), 16, 1024);
      const uint64_t dm0 = tc::sdesc_sw128(saddr(s.kq[0][0][0]), S::kHalf, 1024);
      const uint64_t dt0 = tc::sdesc_sw128(saddr(s.tp[0][0]), kTile, 1024);
      const uint64_t dp0 = tc::sdesc_sw128(saddr(s.tp[0][2]), kTile, 1024);
      auto stop = [&] { return __any_sync(0xffffffffu, s.gave_up) != 0; };
      // do P of the n-th chunk
      auto do_p = [&](int n) {
        const uint64_t dp = dp0 + (n & 1) * (4 * kTile >> 4);
        W(&s.tp_full[n & 1], (n >> 1) & 1);
        W(&s.in_ready, n & 1);
        tc::fence_after_sync();
        if (!stop() && tc::elect_one()) {
          mma_chain<4, true>(tmem + kY, tmem + kAD, 0, dp + lo, 0, id64m, true, 8);
          mma_chain<4, true>(tmem + kY, tmem + kAD, 0, dp, 0, id64m, false, 8);
        }
        __syncwarp();
      };
      int n = 0, end = 0, k = 0;
      // whether there is an n-th chunk (taking the next item for it)
      auto more = [&] {
        if (n < end) return true;
        const Item it = item(k++);
        end = n + (it.bh < 0 ? 0 : it.last - it.first);
        return n < end;
      };
      bool go = more();
      if (go) do_p(0);
      while (go) {
        const uint32_t ph = n & 1, p = n & 1, fill = (n >> 1) & 1;
        const uint64_t dk = dk0 + p * ((KP / 64) * S::kHalf >> 4);
        const uint64_t dm = dm0 + p * ((KP / 64) * S::kHalf >> 4);   // keys; queries a tile on
        const uint64_t dt = dt0 + p * (4 * kTile >> 4);
        W(&s.kq_full[p], fill);
        W(&s.s_ready, ph);
        if (stop()) break;
        tc::fence_after_sync();
        if (tc::elect_one()) {
          mma_chain<KP / 16, false>(tmem + kZ, tmem + kAS, 1, dk, half, id64, true);
          mma_chain<KP / 16, false>(tmem + kZ, tmem + kAS, 0, dk, half, id64, false);
          tc::mma_commit(&s.z_done);
          mma_chain<4, true>(tmem + kW, tmem + kA1, 1, dm + lo, 0, idw, true);
          mma_chain<4, true>(tmem + kW, tmem + kA1, 0, dm + lo, 0, idw, false);
        }
        __syncwarp();
        W(&s.xt_ready, ph);
        if (stop()) break;
        tc::fence_after_sync();
        if (tc::elect_one()) {
          mma_chain<4, true>(tmem + kY, tmem + kZ, 1, dt, 0, id64m, true);
          mma_chain<4, true>(tmem + kY, tmem + kZ, 0, dt + lo, 0, id64m, false);
          mma_chain<4, true>(tmem + kY, tmem + kZ, 0, dt, 0, id64m, false);
          tc::mma_commit(&s.y_done);
        }
        __syncwarp();
        W(&s.w_ready, ph);
        if (stop()) break;
        tc::fence_after_sync();
        if (tc::elect_one()) {
          mma_chain<4, true>(tmem + kW, tmem + kAS, 1, dm, 0, idw, false);
          mma_chain<4, true>(tmem + kW, tmem + kAS, 0, dm, 0, idw, false);
          tc::mma_commit(&s.w_done);
          tc::mma_commit(&s.kq_empty[p]);
          tc::mma_commit(&s.tp_empty[p]);
        }
        __syncwarp();
        ++n;
        go = more();
        if (go) do_p(n);   // (while dS is on its way)
      }
      if (tc::elect_one()) tc::mma_commit(&s.mma_drain);
      __syncwarp();
      drain(&s.mma_drain, 0, &g_status);
    }
  } else if (warp >= kIoWarp) {
    // ---------------- do into TMEM, dY out of it
    SSD_SETREG("inc", "104");
    const int qr = warp & 3, row = qr * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)qr << 21);
    // (the four warps; a wait that gives up, unlike a barrier, lets every warp end)
    auto together = [&](uint32_t phase) {
      warp_arrive(&s.io_sync, lane);
      W(&s.io_sync, phase);
    };
    auto put_do = [&](int n, int none) {   // (none: of unit rows, nothing comes in)
      const int p = n & 1;
      const unsigned char* const dt = s.d[p][row >> 6] + (row & 63) * 2;
      W(&s.d_full[p], (n >> 1) & 1);
      W(&s.vec_full[p], (n >> 1) & 1);
      for (int q = 0; q < 4; ++q) {
        uint32_t u[8], t[16];
        float x[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {   // pairs of tokens
          const unsigned char* at = dt + (q * 16 + 2 * i) * 128;
          u[i] = none ? 0u
                      : *reinterpret_cast<const uint16_t*>(at) |
                            (uint32_t)*reinterpret_cast<const uint16_t*>(at + 128) << 16;
          x[2 * i] = lo_of(u[i]) * a.scale;
          x[2 * i + 1] = hi_of(u[i]) * a.scale;
        }
        tc::tmem_st8(lanes + kAD + q * 8, u);
        scale_by(x, s.vec[p] + kGam * kC + q * 16);
        two_terms(x, t);
        tc::tmem_st16(lanes + kA1 + q * 16, t);
      }
      warp_arrive(&s.d_empty[p], lane);
      warp_arrive(&s.vec_empty[p], lane);
      tc::tmem_st_wait();
      tc::fence_before_sync();
      warp_arrive(&s.in_ready, lane);
    };
    int k = 0;
    Item it = item(k++);
    int r = it.first;   // the chunk, counted from the end
    if (it.bh >= 0) put_do(0, it.unit);
    for (int n = 0; it.bh >= 0; ++n) {
      const int c = nc - 1 - r;
      const int b = it.bh / a.H, h = it.bh % a.H, v0 = it.v0, vr = v0 + row;
      if (warp == kIoWarp && tc::elect_one()) tc::bulk_wait_read();   // the tiles' last copies
      __syncwarp();
      W(&s.y_done, n & 1);
      tc::fence_after_sync();
      together(0);
      unsigned char* const yt = s.y[0][row >> 6];
      for (int q = 0; q < 4; ++q) {
        uint32_t r[16];
        tc::tmem_ld16(lanes + kY + q * 16, r);
        tc::tmem_ld_wait_regs(r);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float f = __uint_as_float(r[i]);
          const bf16 hi = __float2bfloat16_rn(f);
          unsigned char* at = yt + tile_at<64>(q * 16 + i, (row & 63) >> 3) + (row & 7) * 2;
          *reinterpret_cast<bf16*>(at) = hi;
          *reinterpret_cast<bf16*>(at + 2 * kTile) = __float2bfloat16_rn(f - __bfloat162float(hi));
        }
        if (!a.wide_dv && vr < a.V && a.pass != kParts) {   // rows off 16 bytes
          const int64_t t0 = (int64_t)c * kC + q * 16;
          bf16* dst = static_cast<bf16*>(a.dv) + (((int64_t)b * a.L + t0) * a.H + h) * a.V + vr;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (t0 + i < a.L)
              dst[(int64_t)i * a.H * a.V] = __float2bfloat16_rn(__uint_as_float(r[i]));
        }
      }
      tc::fence_before_sync();
      tc::fence_proxy_async_smem();
      together(1);
      if (warp == kIoWarp) {
        if (tc::elect_one()) {
          if (!s.gave_up && a.pass != kParts) {
            // planes [term][channel half][token][64] of the workspace; the first is dv
            unsigned char* to = reinterpret_cast<unsigned char*>(a.dY) +
                                (((int64_t)it.bh * nc + c) * 2 * (a.VP / 64) + v0 / 64) * kTile;
            for (int i = 0; i < 2; ++i)
              asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                               to + (int64_t)i * (a.VP / 64) * kTile),
                           "r"(saddr(s.y[i][0])), "r"(2 * kTile)
                           : "memory");
            if (a.wide_dv)
              for (int i = 0; i < 2; ++i)
                if (v0 + i * 64 < a.V)
                  tc::tma_store_4d(&mv, s.y[0][i], v0 + i * 64, h, c * kC, b);
          }
          tc::bulk_commit();
        }
        __syncwarp();
      }
      if (++r == it.last) {
        it = item(k++);
        r = it.first;
      }
      if (it.bh >= 0) put_do(n + 1, it.unit);   // (what the MMAs read of n's is done as dY is)
    }
    if (warp == kIoWarp && tc::elect_one()) tc::bulk_wait_all();
  } else {
    // ---------------- the chain
    const int qr = warp & 3, part = warp >> 2, row = qr * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)qr << 21);   // this warp's 32 TMEM lanes
    constexpr int SP = KP / 64;                           // pieces of 16 of dS a thread
    float dS[SP][16];
    Item it = {};
    auto put_state = [&](int p, int c) {
      uint32_t t[16];
      two_terms(dS[p], t);
      tc::tmem_st16(lanes + kAS + (part * SP + p) * 16, t);
      if (a.pass != kParts)
        keep_row<KP>(t, a.dS, (int64_t)it.bh * nc + c, it.v0 + row, (part * SP + p) * 16, a);
    };
    auto told = [&](uint64_t* bar) {   // what this warp wrote to TMEM is there
      tc::tmem_st_wait();
      tc::fence_before_sync();
      warp_arrive(bar, lane);
    };
    int rc = 0, slots = 0;   // the chunk, counted from the end
    for (int n = 0, k = 0;; ++n, ++rc) {
      if (rc == it.last) {
        it = item(k++);
        if (it.bh < 0) break;
        rc = it.first;
        if (rc == 0) {
          read_row<SP>(dS, a.dfinal, it.bh, it.v0 + row, part, a);
        } else if (a.pass == kParts) {
#pragma unroll
          for (int p = 0; p < SP; ++p)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              dS[p][i] = it.unit && row == (part * SP + p) * 16 + i ? 1.f : 0.f;
        } else {
          if (lane == 0 && a.pass == kWhole)
            wait_flag(flag_of(a, it), rc / a.seg, &s.gave_up, &g_status);
          __syncwarp();
          read_slot<SP>(dS, a, it, row, part);
        }
#pragma unroll
        for (int p = 0; p < SP; ++p) put_state(p, nc - 1 - rc);
        told(&s.s_ready);
      }
      const uint32_t ph = n & 1;
      const float* vec = s.vec[ph];
      uint32_t r[16], t[16];
      float x[16];
      const int t0 = part * 16;   // the warp's tokens
      W(&s.vec_full[ph], (n >> 1) & 1);
      // dx = beta e^(G_C - G) Z + do P
      W(&s.z_done, ph);
      tc::fence_after_sync();
      tc::tmem_ld16(lanes + kZ + t0, r);
      tc::tmem_ld16(lanes + kY + t0, t);
      tc::tmem_ld_wait_regs(r);
      tc::tmem_ld_wait_regs(t);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 f = *reinterpret_cast<const float4*>(vec + kWrite * kC + t0 + 4 * i);
        fma2(x[4 * i], x[4 * i + 1], __uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]), f.x,
             f.y, __uint_as_float(t[4 * i]), __uint_as_float(t[4 * i + 1]));
        fma2(x[4 * i + 2], x[4 * i + 3], __uint_as_float(r[4 * i + 2]),
             __uint_as_float(r[4 * i + 3]), f.z, f.w, __uint_as_float(t[4 * i + 2]),
             __uint_as_float(t[4 * i + 3]));
      }
      two_terms(x, r);
      tc::tmem_st16(lanes + kZ + t0, r);
      told(&s.xt_ready);
      // -e^G dY
      W(&s.y_done, ph);
      tc::fence_after_sync();
      tc::tmem_ld16(lanes + kY + t0, r);
      tc::tmem_ld_wait_regs(r);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
      scale_by(x, vec + kRead * kC + t0);
      two_terms(x, r);
      tc::tmem_st16(lanes + kAS + t0, r);
      told(&s.w_ready);
      const float through = vec[kVecs * kC];
      warp_arrive(&s.vec_empty[ph], lane);
      // dS = e^(G_C) dS + W
      W(&s.w_done, ph);
      tc::fence_after_sync();
#pragma unroll
      for (int p = 0; p < SP; ++p) {
        tc::tmem_ld16(lanes + kW + (part * SP + p) * 16, r);
        tc::tmem_ld_wait_regs(r);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          fma2(dS[p][2 * i], dS[p][2 * i + 1], dS[p][2 * i], dS[p][2 * i + 1], through, through,
               __uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
        if (rc + 1 < it.last) put_state(p, nc - 2 - rc);
      }
      if (rc + 1 < it.last) {
        told(&s.s_ready);
      } else if (a.pass == kParts) {
        write_slot<SP>(dS, a, it, row, part);
      } else if (rc + 1 < nc) {   // on to the next segment
        if (a.pass == kJoined) continue;
        write_slot<SP>(dS, a, it, row, part);
        warp_arrive(&s.slot_done, lane);
        if (warp == 0) {
          W(&s.slot_done, slots++ & 1);
          if (lane == 0) raise_flag(flag_of(a, it), (rc + 1) / a.seg);
        }
      } else {
        write_row<SP>(dS, a.dinit, it.bh, it.v0 + row, part, a);
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
  CUtensorMap mq, mk, md, mv;
  const TokStride dense = {a.L * a.H * a.V, (int64_t)a.H * a.V};
  if (!token_map(&mq, a.q, a.qcols, a.G, a.L, a.B, a.sq, true) ||
      !token_map(&mk, a.k, a.kcols, a.G, a.L, a.B, a.sk, true) ||
      !token_map(&md, a.dout, a.docols, a.H, a.L, a.B, a.sdo, false))
    return cudaErrorInvalidValue;
  mv = md;
  if (a.wide_dv && !token_map(&mv, a.dv, a.V, a.H, a.L, a.B, dense, true))
    return cudaErrorInvalidValue;
  const int smem = (int)sizeof(Smem<KP>) + 1024;
  cudaError_t e = cudaFuncSetAttribute(
      tc_reverse_kernel<KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  int grid = 0;
  e = start_work(a, &grid, st);
  if (e != cudaSuccess) return e;
  g_launched = true;
  tc_reverse_kernel<KP><<<grid, kThreads, smem, st>>>(mq, mk, md, mv, a);
  return cudaGetLastError();
}
static_assert(sizeof(Smem<128>) + 1024 <= 227 * 1024, "shared memory");

}  // namespace rev

int tc_reverse_status(int reset, cudaStream_t st, int* bits) {
  return read_status(rev::g_status, rev::g_launched, reset, st, bits);
}
cudaError_t launch_tc_reverse(const Args& args, cudaStream_t st) {
  Args a = args;
  if (a.pass == kParts) {
    cudaError_t e = a.KP == 64 ? rev::run<64>(a, st) : rev::run<128>(a, st);
    if (e == cudaSuccess) e = launch_tc_join(a, st);
    if (e == cudaSuccess) e = copy_first(a, &a.dfinal, a.dinit, st);
    if (e != cudaSuccess) return e;
    a.pass = kJoined;
  }
  return a.KP == 64 ? rev::run<64>(a, st) : rev::run<128>(a, st);
}

}  // namespace delta
}  // namespace ssd
