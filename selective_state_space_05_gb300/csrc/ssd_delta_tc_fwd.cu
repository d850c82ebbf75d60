// The gated delta rule's forward on tcgen05 (ssd_delta_tc.cuh says for which
// inputs), one CTA per (batch row, head, 128 channels), chunk after chunk.
//
// Transposed as in ssd_delta_fwd.cu: TMEM lane = channel, columns = tokens or
// dstate.  Per chunk, with S in the registers of eight warps (a row and half of
// dstate a thread) and as two bf16 terms in TMEM:
//   Y | O1 = S [K | Q]^T                 A: S
//   y = v - e^G Y  -> TMEM               the chain's warps
//   X = y T^T                            A: y, over Y's columns
//   w = beta e^(G_C - G) X -> TMEM
//   W = w K, then O2 = X P^T             A: w in S's columns; x over X's columns
//   S = e^(G_C) S + W -> TMEM
// and beside it out = scale e^G O1 + O2 (P holds scale and beta).  K^T and K are
// one tile read in both orders.  Roles, so that only the chain Y - y - X - w - W - S
// is in a chunk's way:
//   warps 0-7    the chain, a quarter of the lanes and half of the columns each
//   warps 8-11   out
//   warps 12-15  the next chunk's T and P (mma.sync: their operands are 16-row
//                blocks in registers, and the tcgen05 pipe is the chain's)
//   warp 16      issues the MMAs;  17: the copies;  18: the chunks' vectors
// Shared and tensor memory: one CTA an SM.
#include "ssd_delta_tc.cuh"

namespace ssd {
namespace delta {
namespace fwd {

constexpr int kChainWarps = 8, kOutWarp = 8, kPrepWarp = 12, kMmaWarp = 16, kLoadWarp = 17,
              kVecWarp = 18;
constexpr int kThreads = 20 * 32;   // (warp 19 fills the last warpgroup)
// Registers a thread: launched with 96, five warps a quadrant of the SM:
// 2 x 128 + 104 + 80 + 40 = 480
#define SSD_SETREG(dir, n) asm volatile("setmaxnreg." dir ".sync.aligned.u32 " n ";")
constexpr int kKQ = 3, kTP = 2;   // stages
// TMEM columns: S's terms (and w's), Y / y, O1, X / x, O2, W
constexpr uint32_t kAS = 0, kR0 = 128, kO1 = 192, kR1 = 256, kO2 = 320, kW = 384;

template <int KP>
struct Smem {
  static constexpr uint32_t kHalf = 2 * kTile;   // 64 columns: 64 rows of K, 64 of Q
  unsigned char kq[kKQ][KP / 64][2][kTile];
  unsigned char v[2][2][kTile];                  // [channel half][token][64], not swizzled; out
  unsigned char tp[kTP][4][kTile];               // T's terms, P's terms
  unsigned char a[2][kTile];                     // the inverse's A, two terms
  float diag[4][kDiag];
  alignas(16) float vec[kTP][vec_floats<kC>()];
  uint64_t kq_full[kKQ], kq_empty[kKQ], v_full[2], v_empty[2], tp_ready[kTP], tp_empty[kTP],
      vec_ready[kTP], vec_empty[kTP];
  uint64_t s_ready, y_done, yt_ready, x_done, w_ready, w_done, o_done, o1_read, o2_read,
      mma_drain;
  uint32_t tmem;
  volatile int gave_up;
};

__device__ int g_status;

template <int KP, bool KEEP>
__global__ void __launch_bounds__(kThreads, 1)
    tc_forward_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo,
                      const __grid_constant__ Args a) {
  extern __shared__ unsigned char raw[];
  using S = Smem<KP>;
  S& s = *reinterpret_cast<S*>(raw + ((1024 - (saddr(raw) & 1023)) & 1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H, kg = h / (a.H / a.G);
  const int v0 = blockIdx.y * 128;
  const int nc = a.nc;
  if (warp == kMmaWarp) tc::tmem_alloc(&s.tmem, 512);
  if (tid == 0) {
    for (int i = 0; i < kKQ; ++i) {
      tc::mbar_init(&s.kq_full[i], 1);
      tc::mbar_init(&s.kq_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s.v_full[i], 1);
      tc::mbar_init(&s.v_empty[i], 1);
      tc::mbar_init(&s.tp_ready[i], 4);
      tc::mbar_init(&s.tp_empty[i], 1);
      tc::mbar_init(&s.vec_ready[i], 1);
      tc::mbar_init(&s.vec_empty[i], kChainWarps + 4);
    }
    tc::mbar_init(&s.s_ready, kChainWarps);
    tc::mbar_init(&s.yt_ready, kChainWarps);
    tc::mbar_init(&s.w_ready, kChainWarps);
    tc::mbar_init(&s.o1_read, 4);
    tc::mbar_init(&s.o2_read, 4);
    tc::mbar_init(&s.y_done, 1);
    tc::mbar_init(&s.x_done, 1);
    tc::mbar_init(&s.w_done, 1);
    tc::mbar_init(&s.o_done, 1);
    tc::mbar_init(&s.mma_drain, 1);
    tc::mbar_fence_init();
    s.gave_up = 0;
  }
  // T's and P's blocks above the diagonal stay zero
  for (int i = tid; i < kTP * 4 * (int)kTile / 16; i += kThreads)
    reinterpret_cast<uint4*>(s.tp)[i] = make_uint4(0, 0, 0, 0);
  tc::fence_proxy_async_smem();
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s.tmem;
  auto W = [&](uint64_t* bar, uint32_t parity) { wait_for(bar, parity, &s.gave_up, &g_status); };

  if (warp >= kMmaWarp) {
    SSD_SETREG("dec", "40");
    if (warp == kLoadWarp) {
      int nk = 0, nv = 0;   // chunks issued
      auto keys = [&] {
        const int st = nk % kKQ;
        if (nk >= kKQ) W(&s.kq_empty[st], (nk / kKQ - 1) & 1);
        if (__any_sync(0xffffffffu, s.gave_up)) return false;
        if (tc::elect_one()) {
          tc::mbar_arrive_expect_tx(&s.kq_full[st], KP / 64 * 2 * kTile);
          for (int i = 0; i < KP / 64; ++i) {
            tc::tma_load_4d(s.kq[st][i][0], &mk, &s.kq_full[st], i * 64, kg, nk * kC, b);
            tc::tma_load_4d(s.kq[st][i][1], &mq, &s.kq_full[st], i * 64, kg, nk * kC, b);
          }
        }
        __syncwarp();
        ++nk;
        return true;
      };
      bool ok = keys();
      while (ok && nv < nc) {   // keys one chunk ahead of values
        if (nk < nc) ok = keys();
        const int vs = nv & 1;
        if (nv >= 2) W(&s.v_empty[vs], (nv / 2 - 1) & 1);
        ok = ok && !__any_sync(0xffffffffu, s.gave_up);
        if (!ok) break;
        if (tc::elect_one()) {
          tc::mbar_arrive_expect_tx(&s.v_full[vs], 2 * kTile);
          for (int i = 0; i < 2; ++i)
            tc::tma_load_4d(s.v[vs][i], &mv, &s.v_full[vs], v0 + i * 64, h, nv * kC, b);
        }
        __syncwarp();
        ++nv;
      }
      // every copy has landed before the CTA ends
      for (int i = nk > kKQ ? nk - kKQ : 0; i < nk; ++i)
        drain(&s.kq_full[i % kKQ], (i / kKQ) & 1, &g_status);
      for (int i = nv > 2 ? nv - 2 : 0; i < nv; ++i)
        drain(&s.v_full[i & 1], (i / 2) & 1, &g_status);
    } else if (warp == kVecWarp) {
      Gates next = load_gates(a, b, h, 0, lane);
      for (int c = 0; c < nc; ++c) {
        float* const vec = s.vec[c & 1];
        if (c >= kTP) W(&s.vec_empty[c & 1], (c / kTP - 1) & 1);
        chunk_vectors(next, vec, lane);
        if (c + 1 < nc) next = load_gates(a, b, h, (int64_t)(c + 1) * kC, lane);
        warp_arrive(&s.vec_ready[c & 1], lane);
        if (KEEP && blockIdx.y == 0) {
          float* const to = a.vec + ((int64_t)bh * nc + c) * vec_floats<kC>();
          for (int i = lane; i < kVecs * kC + 1; i += 32) to[i] = vec[i];
        }
      }
    } else if (warp == kMmaWarp) {
      // (the warp stays converged, one elected lane issuing: descriptors then live
      // in uniform registers)
      constexpr uint32_t id64 = tc::idesc_bf16(128, 64, false, false);
      constexpr uint32_t id128 = tc::idesc_bf16(128, 128, false, false);
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
      for (int c = 0; c < nc; ++c) {
        const uint32_t ph = c & 1, tp = c & 1;
        const uint64_t dk = dk0 + st * ((KP / 64) * S::kHalf >> 4);
        const uint64_t dm = dm0 + st * ((KP / 64) * S::kHalf >> 4);
        const uint64_t dt = dt0 + tp * (4 * kTile >> 4), dp = dp0 + tp * (4 * kTile >> 4);
        W(&s.kq_full[st], kq_ph);
        if (c > 0) W(&s.o1_read, ph ^ 1);
        W(&s.s_ready, ph);
        if (stop()) break;
        tc::fence_after_sync();
        if (tc::elect_one()) {
          mma_chain<KP / 16, false>(tmem + kR0, tmem + kAS, 1, dk, half, id128, true);
          mma_chain<KP / 16, false>(tmem + kR0, tmem + kAS, 0, dk, half, id128, false);
          tc::mma_commit(&s.y_done);
        }
        __syncwarp();
        W(&s.tp_ready[tp], (c >> 1) & 1);
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
        }
        __syncwarp();
        if (c > 0) W(&s.o2_read, ph ^ 1);
        if (stop()) break;
        tc::fence_after_sync();
        if (tc::elect_one()) {
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
  } else if (warp >= kPrepWarp) {
    // ---------------- the chunks' T and P
    SSD_SETREG("dec", "80");
    const int w = warp - kPrepWarp, ptid = tid - kPrepWarp * 32;
    for (int c = 0; c < nc; ++c) {
      const int st = c % kKQ, tp = c & 1;
      const float* const vec = s.vec[tp];
      const bool keys = w < 2;
      const uint32_t ba = saddr(s.kq[st][0][keys ? 0 : 1]), bk = saddr(s.kq[st][0][0]);
      float x[10][4];
      W(&s.kq_full[st], (c / kKQ) & 1);
      if (w & 1) pair_products<KP, true>(x, ba, bk, S::kHalf, lane);
      else pair_products<KP, false>(x, ba, bk, S::kHalf, lane);
      W(&s.vec_ready[tp], (c >> 1) & 1);
      if (c >= kTP) W(&s.tp_empty[tp], (c / kTP - 1) & 1);
      if (KEEP && ptid == 0) tc::bulk_wait_read();
      named_sync(2, 128);   // all four are past the chunk before
      unsigned char* const to = keys ? s.a[0] : s.tp[tp][2];
      if (w & 1) pair_decays<true>(x, vec, keys, a.scale, to, s.diag[0], lane);
      else pair_decays<false>(x, vec, keys, a.scale, to, s.diag[0], lane);
      named_sync(2, 128);
      invert(s.tp[tp][0], s.a[0], s.diag[0], w, lane, 2);
      tc::fence_proxy_async_smem();
      if (KEEP) {
        named_sync(2, 128);
        if (blockIdx.y == 0 && ptid == 0) {
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                           reinterpret_cast<unsigned char*>(a.T) + ((int64_t)bh * nc + c) * 4 * kTile),
                       "r"(saddr(s.tp[tp][0])), "r"(4 * kTile)
                       : "memory");
          tc::bulk_commit();
        }
      }
      warp_arrive(&s.tp_ready[tp], lane);
    }
    if (KEEP && ptid == 0) tc::bulk_wait_all();
  } else if (warp >= kOutWarp) {
    // ---------------- out = scale e^G O1 + O2, over v's tile
    SSD_SETREG("inc", "104");
    const int qr = warp & 3, row = qr * 32 + lane, vr = v0 + row;
    const uint32_t lanes = tmem + ((uint32_t)qr << 21);
    for (int c = 0; c < nc; ++c) {
      const uint32_t ph = c & 1;
      const float* gam = s.vec[ph] + kGam * kC;
      unsigned char* const vt = s.v[ph][row >> 6] + (row & 63) * 2;
      uint32_t o1[4][16];
      W(&s.x_done, ph);   // O1 is done as X is
      tc::fence_after_sync();
#pragma unroll
      for (int p = 0; p < 4; ++p) tc::tmem_ld16(lanes + kO1 + p * 16, o1[p]);
#pragma unroll
      for (int p = 0; p < 4; ++p) tc::tmem_ld_wait_regs(o1[p]);
      tc::fence_before_sync();
      warp_arrive(&s.o1_read, lane);
      W(&s.o_done, ph);
      tc::fence_after_sync();
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        uint32_t r[16];
        float x[16];
        tc::tmem_ld16(lanes + kO2 + p * 16, r);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(o1[p][i]) * a.scale;
        scale_by(x, gam + p * 16);
        tc::tmem_ld_wait_regs(r);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] += __uint_as_float(r[i]);
        if (a.wide_out) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            *reinterpret_cast<bf16*>(vt + (p * 16 + i) * 128) = __float2bfloat16_rn(x[i]);
        } else if (a.out && vr < a.V) {   // rows off 16 bytes
          const int64_t t0 = (int64_t)c * kC + p * 16;
          bf16* dst = static_cast<bf16*>(a.out) + (((int64_t)b * a.L + t0) * a.H + h) * a.V + vr;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (t0 + i < a.L) dst[(int64_t)i * a.H * a.V] = __float2bfloat16_rn(x[i]);
        }
      }
      tc::fence_before_sync();
      warp_arrive(&s.o2_read, lane);
      warp_arrive(&s.vec_empty[ph], lane);
      tc::fence_proxy_async_smem();
      named_sync(1, 128);
      if (warp == kOutWarp) {
        if (tc::elect_one()) {
          if (a.wide_out && !s.gave_up)
            for (int i = 0; i < 2; ++i)
              if (v0 + i * 64 < a.V) tc::tma_store_4d(&mo, s.v[ph][i], v0 + i * 64, h, c * kC, b);
          tc::bulk_commit();
          tc::bulk_wait_read();
          tc::mbar_arrive(&s.v_empty[ph]);
        }
        __syncwarp();
      }
    }
    if (warp == kOutWarp && tc::elect_one()) tc::bulk_wait_all();
  } else {
    // ---------------- the chain
    SSD_SETREG("inc", "128");
    const int qr = warp & 3, hf = warp >> 2, row = qr * 32 + lane, vr = v0 + row;
    const uint32_t lanes = tmem + ((uint32_t)qr << 21);   // this warp's 32 TMEM lanes
    constexpr int SP = KP / 32;                           // pieces of 16 of S a thread
    const bool live = vr < a.V;
    float S0[SP][16];
    {
      const float* src = a.init ? a.init + ((int64_t)bh * a.V + (live ? vr : 0)) * a.K : nullptr;
#pragma unroll
      for (int p = 0; p < SP; ++p)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int k = (hf * SP + p) * 16 + i;
          S0[p][i] = src && live && k < a.K ? src[k] : 0.f;
        }
    }
    // A piece of S as terms to TMEM (and to memory, as chunk c's first state)
    auto put_state = [&](int p, int c) {
      uint32_t t[16];
      two_terms(S0[p], t);
      tc::tmem_st16(lanes + kAS + (hf * SP + p) * 16, t);
      if (KEEP) {
        // planes [term][dstate half][row][64], swizzled as the tiles
        const int k = (hf * SP + p) * 16;
        unsigned char* at = reinterpret_cast<unsigned char*>(a.S0) +
                            (((int64_t)bh * nc + c) * 2 * (KP / 64) + (k >> 6)) * a.VP * 128 +
                            (int64_t)vr * 128;
        const int64_t plane = (int64_t)a.VP * KP * 2;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int unit = (((k & 63) >> 3) + i) ^ (vr & 7);
          *reinterpret_cast<uint4*>(at + unit * 16) =
              make_uint4(t[4 * i], t[4 * i + 1], t[4 * i + 2], t[4 * i + 3]);
          *reinterpret_cast<uint4*>(at + plane + unit * 16) =
              make_uint4(t[8 + 4 * i], t[9 + 4 * i], t[10 + 4 * i], t[11 + 4 * i]);
        }
      }
    };
    auto told = [&](uint64_t* bar) {   // what this warp wrote to TMEM is there
      tc::tmem_st_wait();
      tc::fence_before_sync();
      warp_arrive(bar, lane);
    };
#pragma unroll
    for (int p = 0; p < SP; ++p) put_state(p, 0);
    told(&s.s_ready);
    for (int c = 0; c < nc; ++c) {
      const uint32_t ph = c & 1;
      const float* vec = s.vec[ph];
      const unsigned char* const vt = s.v[ph][row >> 6] + (row & 63) * 2;
      uint32_t r[2][16];
      // y = v - e^G Y
      W(&s.v_full[ph], (c >> 1) & 1);
      W(&s.vec_ready[ph], (c >> 1) & 1);
      W(&s.y_done, ph);
      tc::fence_after_sync();
#pragma unroll
      for (int p = 0; p < 2; ++p) tc::tmem_ld16(lanes + kR0 + (hf * 2 + p) * 16, r[p]);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int t0 = (hf * 2 + p) * 16;
        float x[16];
        tc::tmem_ld_wait_regs(r[p]);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = -__uint_as_float(r[p][i]);
        scale_by(x, vec + kGam * kC + t0);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          x[i] += __uint_as_float(
              (uint32_t)*reinterpret_cast<const uint16_t*>(vt + (t0 + i) * 128) << 16);
        two_terms(x, r[p]);
        tc::tmem_st16(lanes + kR0 + t0, r[p]);
      }
      told(&s.yt_ready);
      // x's terms, and w = beta e^(G_C - G) x
      W(&s.x_done, ph);
      tc::fence_after_sync();
#pragma unroll
      for (int p = 0; p < 2; ++p) tc::tmem_ld16(lanes + kR1 + (hf * 2 + p) * 16, r[p]);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int t0 = (hf * 2 + p) * 16;
        float x[16];
        uint32_t t[16];
        tc::tmem_ld_wait_regs(r[p]);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[p][i]);
        two_terms(x, t);
        tc::tmem_st16(lanes + kR1 + t0, t);
        scale_by(x, vec + kBeta * kC + t0);
        scale_by(x, vec + kOnto * kC + t0);
        two_terms(x, r[p]);
        tc::tmem_st16(lanes + kAS + t0, r[p]);
        if (KEEP) {
          // planes [term][channel half][token][64], swizzled
          unsigned char* base = reinterpret_cast<unsigned char*>(a.X) +
                                ((int64_t)bh * nc + c) * 2 * kC * a.VP * 2 +
                                (int64_t)(vr >> 6) * kTile;
          const int64_t plane = (int64_t)kC * a.VP * 2;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            unsigned char* at = base + tile_at<64>(t0 + i, (vr & 63) >> 3) + (vr & 7) * 2;
            const int sh = 16 * (i & 1);
            *reinterpret_cast<uint16_t*>(at) = (uint16_t)(t[i >> 1] >> sh);
            *reinterpret_cast<uint16_t*>(at + plane) = (uint16_t)(t[8 + (i >> 1)] >> sh);
          }
        }
      }
      told(&s.w_ready);
      const float through = vec[kVecs * kC];
      warp_arrive(&s.vec_empty[ph], lane);
      // S = e^(G_C) S + W
      W(&s.w_done, ph);
      tc::fence_after_sync();
#pragma unroll
      for (int p = 0; p < SP; ++p) {
        if (p % 2 == 0) {
          tc::tmem_ld16(lanes + kW + (hf * SP + p) * 16, r[0]);
          if (p + 1 < SP) tc::tmem_ld16(lanes + kW + (hf * SP + p + 1) * 16, r[1]);
        }
        tc::tmem_ld_wait_regs(r[p & 1]);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          S0[p][i] = fmaf(through, S0[p][i], __uint_as_float(r[p & 1][i]));
        if (c + 1 < nc) put_state(p, c + 1);
      }
      told(&s.s_ready);
    }
    if (a.final && live) {
      float* dst = a.final + ((int64_t)bh * a.V + vr) * a.K;
#pragma unroll
      for (int p = 0; p < SP; ++p)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int k = (hf * SP + p) * 16 + i;
          if (k < a.K) dst[k] = S0[p][i];
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
  const int smem = (int)sizeof(Smem<KP>) + 1024;
  const cudaError_t e = cudaFuncSetAttribute(
      tc_forward_kernel<KP, KEEP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(a.B * a.H), (unsigned)((a.V + 127) / 128));
  tc_forward_kernel<KP, KEEP><<<grid, kThreads, smem, st>>>(mq, mk, mv, mo, a);
  return cudaGetLastError();
}
static_assert(sizeof(Smem<128>) + 1024 <= 227 * 1024, "shared memory");

}  // namespace fwd

// Status bits of the launches that gave up a wait (host; ssd_scan_status).
int tc_forward_status(int reset, cudaStream_t st, int* bits) {
  return read_status(fwd::g_status, reset, st, bits);
}

cudaError_t launch_tc_forward(const Args& a, cudaStream_t st) {
  if (a.KP == 64) return a.S0 ? fwd::run<64, true>(a, st) : fwd::run<64, false>(a, st);
  return a.S0 ? fwd::run<128, true>(a, st) : fwd::run<128, false>(a, st);
}

}  // namespace delta
}  // namespace ssd
