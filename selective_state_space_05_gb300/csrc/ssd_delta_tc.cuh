// What the gated delta rule's tcgen05 kernels share: bounded waits, tensor maps,
// operands in TMEM, and a chunk's triangular inverse.
//
// These kernels take bf16 tensors whose rows lie on 16 bytes (others are packed
// first), 128 headdim channels a CTA: the state's rows are TMEM lanes, so that every
// product of a chunk has its fp32 factor as A operand in TMEM (two bf16 terms) and
// keys, queries or the chunk's matrices as B operand in shared memory, as 64-column
// tiles with the 128-byte swizzle.  (Measured for M = 128, K = 16: 44, 64 and 128
// cycles for N = 64, 128 and 256, and 200 from a commit to the waiting warps; M = 64
// takes as long as 128.)
#pragma once

#include <cudaTypedefs.h>

#include <atomic>

#include "ssd_delta.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace delta {

// A role's registers: the roles' sum stays within what the CTA was launched with.
#define SSD_SETREG(dir, n) asm volatile("setmaxnreg." dir ".sync.aligned.u32 " n ";")

constexpr int kC = 64;              // tokens a chunk
constexpr uint32_t kTile = kC * 128;   // bytes of 64 rows of 64 columns
enum { kErrWait = 1, kErrDrain = 4 };   // bits of the status word (ssd_scan_status)

// A wait for an mbarrier's phase that gives up after kTries polls (each of which
// suspends the thread for a while: they take seconds, and no wait takes a
// millisecond), or at once when the CTA has given up before: it then records that
// in `gave_up` (shared) and in the device's status word, and the caller goes on
// without what it waited for (every later wait returns at once, nothing more is
// issued, and the launch ends).  Short, since every role's loop has several.
constexpr uint32_t kTries = 4000000;
__device__ __forceinline__ void wait_for(uint64_t* bar, uint32_t parity, volatile int* gave_up,
                                         int* status) {
  for (uint32_t i = 0; !tc::mbar_try_wait(bar, parity); ++i) {
    if (*gave_up) return;
    if (i == kTries) {
      *gave_up = 1;
      atomicOr(status, kErrWait);
    }
  }
}
// At the end of a launch, for copies or MMAs in flight: not cut short.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity, int* status) {
  for (uint32_t i = 0; !tc::mbar_try_wait_sleep(bar, parity, 10000); ++i)
    if (i == kTries) {
      atomicOr(status, kErrDrain);
      return;
    }
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// A warp's arrival for what all its lanes have done.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) tc::mbar_arrive(bar);
}

// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
}
__device__ __forceinline__ void fma2(float& x, float& y, float a0, float a1, float b0, float b1,
                                     float c0, float c1) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d) : "l"(pair_of(a0, a1)), "l"(pair_of(b0, b1)), "l"(pair_of(c0, c1)));
  unpair(d, x, y);
}
__device__ __forceinline__ void mul2(float& x, float& y, float b0, float b1) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair_of(x, y)), "l"(pair_of(b0, b1)));
  unpair(d, x, y);
}
__device__ __forceinline__ void add2p(float& x, float& y, float b0, float b1) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair_of(x, y)), "l"(pair_of(b0, b1)));
  unpair(d, x, y);
}
// 16 values as two terms in pairs: words 0-7 the first, 8-15 the second.  A K step
// of 16 columns of an A operand stands so in 16 TMEM columns.
__device__ __forceinline__ void two_terms(const float (&v)[16], uint32_t (&t)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float x = v[2 * i], y = v[2 * i + 1];
    t[i] = pack2_part(x, y);
    add2p(x, y, __uint_as_float((t[i] << 16) ^ 0x80000000u),
          __uint_as_float((t[i] & 0xFFFF0000u) ^ 0x80000000u));
    t[8 + i] = pack2(x, y);
  }
}
// Products with 16 factors in shared memory (16-byte aligned).
__device__ __forceinline__ void scale_by(float (&x)[16], const float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 w = *reinterpret_cast<const float4*>(f + 4 * i);
    mul2(x[4 * i], x[4 * i + 1], w.x, w.y);
    mul2(x[4 * i + 2], x[4 * i + 3], w.z, w.w);
  }
}
// D (+)= A B over A's K steps [0, STEPS), for term `ta` of A and the tile(s) at b: a
// K-major descriptor (32 bytes a step inside 64 columns, `half` 16-byte units to
// the next 64) or an MN-major one (16 rows a step).
// (a_step: TMEM columns a step of A takes, 8 for one with a single term.)
template <int STEPS, bool MN>
__device__ __forceinline__ void mma_chain(uint32_t d, uint32_t a, int ta, uint64_t b, uint32_t half,
                                          uint32_t idesc, bool fresh, int a_step = 16) {
#pragma unroll
  for (int ks = 0; ks < STEPS; ++ks)
    tc::mma_ts(d, a + ks * a_step + ta * 8,
               b + (MN ? (uint32_t)ks * 128u : (uint32_t)(ks >> 2) * half + (uint32_t)(ks & 3) * 2u),
               idesc, !(fresh && ks == 0));
}

// SP pieces of 16 of a row of a [B, H, V, K] fp32 state, from column part * SP * 16
// on; zeros where there is none.
template <int SP>
__device__ __forceinline__ void read_row(float (&x)[SP][16], const float* state, int bh, int vr,
                                         int part, const Args& a) {
  const float* row = state + ((int64_t)bh * a.V + vr) * a.K;
  const bool wide = a.K % 4 == 0 && ((uintptr_t)state & 15) == 0;
#pragma unroll
  for (int p = 0; p < SP; ++p)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = (part * SP + p) * 16 + 4 * i;
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (state && vr < a.V) {
        if (wide) {
          if (k < a.K) f = *reinterpret_cast<const float4*>(row + k);
        } else {
          if (k < a.K) f.x = row[k];
          if (k + 1 < a.K) f.y = row[k + 1];
          if (k + 2 < a.K) f.z = row[k + 2];
          if (k + 3 < a.K) f.w = row[k + 3];
        }
      }
      x[p][4 * i] = f.x;
      x[p][4 * i + 1] = f.y;
      x[p][4 * i + 2] = f.z;
      x[p][4 * i + 3] = f.w;
    }
}
template <int SP>
__device__ __forceinline__ void write_row(const float (&x)[SP][16], float* state, int bh, int vr,
                                          int part, const Args& a) {
  if (!state || vr >= a.V) return;
  float* row = state + ((int64_t)bh * a.V + vr) * a.K;
  const bool wide = a.K % 4 == 0 && ((uintptr_t)state & 15) == 0;
#pragma unroll
  for (int p = 0; p < SP; ++p)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = (part * SP + p) * 16 + 4 * i;
      if (wide) {
        if (k < a.K)
          *reinterpret_cast<float4*>(row + k) =
              make_float4(x[p][4 * i], x[p][4 * i + 1], x[p][4 * i + 2], x[p][4 * i + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (k + e < a.K) row[k + e] = x[p][4 * i + e];
      }
    }
}
// ------------------------------------------------------------------ work
// A CTA takes (segment, head, 128 channels) items by tickets, in segments' order, so
// that heads that do not divide into the SMs leave none idle: an item's state comes
// from the one a whole round of heads earlier, through the L2.  The predecessor of a
// ticket that was taken has been taken too: whatever else runs on the GPU, waiting
// for it ends.
struct Item {
  int bh, v0, first, last;   // head, channel, chunks [first, last)
  int slot;                  // where its state comes from or goes to (kParts, kJoined)
  int unit;                  // from unit rows, without values
};
__device__ __forceinline__ Item item_of(const Args& a, int ticket) {
  const int vb = (a.V + 127) / 128, n = a.B * a.H * vb;
  Item i = {-1, 0, 0, 0, 0, 0};
  int seg = 0;
  if (a.pass == kParts && ticket >= n * (a.segs - 1)) {
    // M of the segments between the first and the last, behind the W
    const int t = ticket - n * (a.segs - 1);
    if (t >= a.B * a.H * (a.segs - 2)) return i;
    i.bh = t % (a.B * a.H);
    seg = t / (a.B * a.H) + 1;
    i.unit = 1;
    i.slot = ticket;
  } else {
    if (ticket >= n * (a.pass == kParts ? a.segs - 1 : a.segs)) return i;
    const int r = ticket % n;
    seg = ticket / n;
    i.bh = r / vb;
    i.v0 = r % vb * 128;
    i.slot = a.pass == kJoined ? ticket - n : ticket;
  }
  i.first = seg * a.seg;
  i.last = min(i.first + a.seg, a.nc);
  return i;
}
// Two items ahead in shared memory.
struct Items {
  Item item[2];
  uint64_t full[2], empty[2];
};
// Waits for an item's predecessor (one warp), and lets its successor go on (after a
// barrier of the warps that wrote its state).
__device__ __forceinline__ int* flag_of(const Args& a, const Item& i) {
  return a.ctrl + 1 + i.bh * ((a.V + 127) / 128) + i.v0 / 128;
}
__device__ __forceinline__ void wait_flag(const int* flag, int want, volatile int* gave_up,
                                          int* status) {
  for (uint32_t n = 0;; ++n) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
    if (v >= want || *gave_up) break;
    if (n == kTries) {
      *gave_up = 1;
      atomicOr(status, kErrWait);
    }
    __nanosleep(100);
  }
}
__device__ __forceinline__ void raise_flag(int* flag, int to) {
  __threadfence();
  asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(flag), "r"(to) : "memory");
}
// A row of a state between segments: [head, 128 channels][16 columns][4 of them][row],
// a warp's rows side by side.
__device__ __forceinline__ int slot_of(const Args& a, const Item& it) {
  return a.pass == kWhole ? it.bh * ((a.V + 127) / 128) + it.v0 / 128 : it.slot;
}
template <int SP>
__device__ __forceinline__ void read_slot(float (&x)[SP][16], const Args& a, const Item& it, int row,
                                          int part) {
  const float4* p =
      reinterpret_cast<const float4*>(a.slots) + (int64_t)slot_of(a, it) * 32 * a.KP + row;
#pragma unroll
  for (int k = 0; k < SP; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float4 f;
      asm volatile("ld.relaxed.gpu.global.v4.f32 {%0,%1,%2,%3}, [%4];"
                   : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
                   : "l"(p + ((part * SP + k) * 4 + i) * 128) : "memory");
      x[k][4 * i] = f.x;
      x[k][4 * i + 1] = f.y;
      x[k][4 * i + 2] = f.z;
      x[k][4 * i + 3] = f.w;
    }
}
template <int SP>
__device__ __forceinline__ void write_slot(const float (&x)[SP][16], const Args& a, const Item& it,
                                           int row, int part) {
  float4* p = reinterpret_cast<float4*>(a.slots) + (int64_t)slot_of(a, it) * 32 * a.KP + row;
#pragma unroll
  for (int k = 0; k < SP; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[((part * SP + k) * 4 + i) * 128] =
          make_float4(x[k][4 * i], x[k][4 * i + 1], x[k][4 * i + 2], x[k][4 * i + 3]);
}

// 16 columns from k on of row vr of chunk id's state, as terms: planes [block of 128
// rows][term][8 columns][row], so that a warp's rows lie side by side and a block is
// an MMA operand's core matrices (no swizzle).
template <int KP>
__device__ __forceinline__ void keep_row(const uint32_t (&t)[16], bf16* planes, int64_t id, int vr,
                                         int k, const Args& a) {
  uint4* at = reinterpret_cast<uint4*>(planes) +
              (((id * (a.VP / 128) + (vr >> 7)) * 2) * (KP / 8) + (k >> 3)) * 128 + (vr & 127);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    at[i * 128] = make_uint4(t[4 * i], t[4 * i + 1], t[4 * i + 2], t[4 * i + 3]);
    at[(KP / 8 + i) * 128] = make_uint4(t[8 + 4 * i], t[9 + 4 * i], t[10 + 4 * i], t[11 + 4 * i]);
  }
}
// Descriptor of such a block (MN-major without swizzle): groups of eight rows along
// K 128 bytes apart, of eight columns along MN 2048.
__device__ __forceinline__ uint64_t sdesc_rows(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 16 |
         (uint64_t)(2048 >> 4) << 32 | 1ull << 46;
}

// ------------------------------------------------------------------ a chunk's matrices
// Transposes an 8 x 8 block of bf16 held as an accumulator's packed pairs.
__device__ __forceinline__ uint32_t trans8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// A 16 x 16 block [m][n] in two accumulator tiles, negated and transposed, as two
// terms to rows `row` .. and columns `col` .. of a tile's planes.
__device__ __forceinline__ void store_block_t(const float (&x)[4], const float (&y)[4],
                                              unsigned char* base, int row, int col, int lane) {
  const float* v[2] = {x, y};
#pragma unroll
  for (int j = 0; j < 2; ++j)        // eight rows of the result
#pragma unroll
    for (int r = 0; r < 2; ++r) {    // eight of its columns
      uint32_t w[2];
      split2<2>(-v[j][2 * r], -v[j][2 * r + 1], w);
      const uint32_t at = tile_at<64>(row + 8 * j + (lane >> 2), (col + 8 * r) >> 3) + (lane & 3) * 4;
#pragma unroll
      for (int t = 0; t < 2; ++t)
        *reinterpret_cast<uint32_t*>(base + t * kTile + at) = trans8(w[t]);
    }
}
constexpr int kDiag = 16 * 16;   // floats of a diagonal block's transpose

// T = (I + A)^-1 for strictly lower A [64][64], by four warps (named barrier `id`):
// A's blocks below the diagonal as planes, its diagonal blocks transposed in fp32;
// T as planes, whose blocks above the diagonal are zero already.  The diagonal
// blocks by substitution, a column a lane; then -T_ii A_ij T_jj, doubling the side
// twice, transposed, so that each product's result is the next one's A operand.
__device__ __forceinline__ void invert(unsigned char* t, const unsigned char* a,
                                       const float* diag, int w, int lane, int id) {
  {
    const float* d = diag + w * kDiag;
    const int c = lane & 15;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i == c ? 1.f : 0.f;
#pragma unroll
    for (int j = 0; j < 15; ++j) {
#pragma unroll
      for (int q = (j + 1) / 4; q < 4; ++q) {
        const float4 f = *reinterpret_cast<const float4*>(d + j * 16 + 4 * q);
        const float col[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * q + e > j) x[4 * q + e] = fmaf(-col[e], x[j], x[4 * q + e]);
      }
    }
    if (lane < 16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        uint32_t h[2];
        split2<2>(x[i], 0.f, h);
        unsigned char* p = t + tile_at<64>(w * 16 + i, (w * 16 + c) >> 3) + (c & 7) * 2;
        *reinterpret_cast<uint16_t*>(p) = (uint16_t)h[0];
        *reinterpret_cast<uint16_t*>(p + kTile) = (uint16_t)h[1];
      }
    }
  }
  named_sync(id, 128);
  if (w < 2) {
    const int r = 32 * w;
    uint32_t f[2][4];
    float y[2][4], z[2][4];
    zero(y);
    zero(z);
#pragma unroll
    for (int i = 0; i < 2; ++i) a_from_t(f[i], block_at<64>(saddr(t) + i * kTile, r, r, lane));
    mma_pair<2, 2, false>(y[0], y[1], f, blockn_at<64>(saddr(a), r + 16, r, lane), kTile);
    a_from<2>(y[0], y[1], f);
    mma_pair<2, 2, false>(z[0], z[1], f, blockn_at<64>(saddr(t), r + 16, r + 16, lane), kTile);
    store_block_t(z[0], z[1], t, r + 16, r, lane);
  }
  named_sync(id, 128);
  {
    const int m = (w & 1) * 16, n = 32 + (w >> 1) * 16;
    uint32_t f[2][4];
    float y[4][4], z[2][4];
    zero(y);
    zero(z);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        a_from_t(f[i], block_at<64>(saddr(t) + i * kTile, ks * 16, m, lane));
#pragma unroll
      for (int p = 0; p < 2; ++p)
        mma_pair<2, 2, false>(y[2 * p], y[2 * p + 1], f,
                              blockn_at<64>(saddr(a), 32 + p * 16, ks * 16, lane), kTile);
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      a_from<2>(y[2 * ks], y[2 * ks + 1], f);
      mma_pair<2, 2, false>(z[0], z[1], f, blockn_at<64>(saddr(t), n, 32 + ks * 16, lane), kTile);
    }
    store_block_t(z[0], z[1], t, n, m, lane);
  }
}

// A chunk's vectors by one warp, two tokens a lane; g0.. are the lane's tokens'.
struct Gates {
  float g[2], be[2];
  int reset[2];
};
__device__ __forceinline__ Gates load_gates(const Args& a, int b, int h, int64_t t0, int lane) {
  Gates x;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int64_t t = t0 + lane * 2 + e;
    x.g[e] = x.be[e] = 0.f;
    x.reset[e] = 0;
    if (t < a.L) {
      const int64_t at = ((int64_t)b * a.L + t) * a.H + h;
      x.g[e] = a.g[at];
      x.be[e] = a.beta[at];
      if (a.seq && t > 0) {
        const int32_t* q = a.seq + (int64_t)b * a.L + t;
        x.reset[e] = q[0] != q[-1];
      }
    }
  }
  return x;
}
// A sum kept as two floats: the larger and what its rounding left (fp64 would be
// as exact, but its pipe takes ten times as long here).
struct Sum2 {
  float hi, lo;
};
__device__ __forceinline__ Sum2 add2(Sum2 a, Sum2 b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  const float e = ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo);
  Sum2 r;
  r.hi = s + e;
  r.lo = e - (r.hi - s);
  return r;
}
__device__ __forceinline__ Sum2 shfl_up2(Sum2 a, int off) {
  return {__shfl_up_sync(0xffffffffu, a.hi, off), __shfl_up_sync(0xffffffffu, a.lo, off)};
}
// kGhi, kGlo: G log2(e) in two floats, so that a decay is one ex2 of a difference.
__device__ __forceinline__ void chunk_vectors(Gates x, float* vec, int lane) {
  Sum2 s[2], run = {0.f, 0.f};
  int seg[2], cnt = 0;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (x.g[e] < kReset) {
      x.g[e] = 0.f;
      x.reset[e] = 1;
    }
    run = add2(run, {x.g[e], 0.f});
    cnt += x.reset[e];
    s[e] = run;
    seg[e] = cnt;
  }
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Sum2 v = shfl_up2(run, off);
    const int n = __shfl_up_sync(0xffffffffu, cnt, off);
    if (lane >= off) {
      run = add2(v, run);
      cnt += n;
    }
  }
  const Sum2 total = {__shfl_sync(0xffffffffu, run.hi, 31), __shfl_sync(0xffffffffu, run.lo, 31)};
  const int segs = __shfl_sync(0xffffffffu, cnt, 31);
  Sum2 before = shfl_up2(run, 1);
  int cbefore = __shfl_up_sync(0xffffffffu, cnt, 1);
  if (lane == 0) {
    before = {0.f, 0.f};
    cbefore = 0;
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = lane * 2 + e;
    const Sum2 G = add2(before, s[e]);
    const int sg = cbefore + seg[e];
    const float rest = (total.hi - G.hi) + (total.lo - G.lo);
    // G log2(e): the product's rounding and the factor's own tail go to the low part
    const float hi = G.hi * kLog2e;
    const float lo = fmaf(G.hi, kLog2e, -hi) + fmaf(G.hi, 1.925963033500e-8f, G.lo * kLog2e);
    vec[kGam * kC + i] = sg == 0 ? expf(G.hi) : 0.f;
    const float onto = sg == segs ? expf(rest) : 0.f;
    vec[kOnto * kC + i] = onto;
    vec[kBeta * kC + i] = x.be[e];
    vec[kRead * kC + i] = sg == 0 ? -expf(G.hi) : 0.f;
    vec[kWrite * kC + i] = onto * x.be[e];
    vec[kGhi * kC + i] = hi;
    vec[kGlo * kC + i] = lo;
    vec[kSeg * kC + i] = (float)sg;
  }
  if (lane == 0) vec[kVecs * kC] = segs == 0 ? expf(total.hi) : 0.f;
}

// Two warps of four for k k^T, two for q k^T (64 x 64, lower triangles): a warp has
// the rows of 16 from 3 and 0 (ODD: 2 and 1), five blocks of 16 x 16, block q in
// x[2q], x[2q + 1].  ba: the first 64 columns' rows of A, bk: keys' (`next` bytes
// to the next 64 columns).
template <int KP, bool ODD>
__device__ __forceinline__ void pair_products(float (&x)[10][4], uint32_t ba, uint32_t bk,
                                              uint32_t next, int lane) {
  constexpr int r0 = ODD ? 2 : 3, r1 = ODD ? 1 : 0;
  zero(x);
#pragma unroll
  for (int ks = 0; ks < KP / 16; ++ks) {
    const uint32_t off = (ks >> 2) * next;
    uint32_t f0[4], f1[4], k[r0 + 1][4];
    ldsm(f0, block_at<64>(ba + off, r0 * 16, (ks & 3) * 16, lane));
    ldsm(f1, block_at<64>(ba + off, r1 * 16, (ks & 3) * 16, lane));
#pragma unroll
    for (int n = 0; n <= r0; ++n) ldsm(k[n], blockn_at<64>(bk + off, n * 16, (ks & 3) * 16, lane));
#pragma unroll
    for (int n = 0; n <= r0; ++n) {
      mma(x[2 * n], f0, k[n][0], k[n][1]);
      mma(x[2 * n + 1], f0, k[n][2], k[n][3]);
    }
#pragma unroll
    for (int n = 0; n <= r1; ++n) {
      mma(x[2 * (r0 + 1 + n)], f1, k[n][0], k[n][1]);
      mma(x[2 * (r0 + 1 + n) + 1], f1, k[n][2], k[n][3]);
    }
  }
}
// Those products with their decays: A = strictly lower D k k^T beta_j into planes
// (its diagonal blocks transposed to diag), or P = lower D q k^T scale beta_j, as
// terms.  RESETS: whether a state starts anew within the chunk.
template <bool ODD, bool RESETS>
__device__ __forceinline__ void pair_decays(const float (&x)[10][4], const float* vec, bool keys,
                                            float scale, unsigned char* planes, float* diag,
                                            int lane) {
  constexpr int r0 = ODD ? 2 : 3, r1 = ODD ? 1 : 0;
  const int g = lane >> 2, t = lane & 3;
  const float neg = __int_as_float(0xff800000), f = keys ? 1.f : scale;
  float hi[4], lo[4], sg[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {   // the two rows of r0, the two of r1
    const int i = (r < 2 ? r0 : r1) * 16 + g + 8 * (r & 1);
    hi[r] = vec[kGhi * kC + i];
    lo[r] = vec[kGlo * kC + i];
    sg[r] = RESETS ? vec[kSeg * kC + i] : 0.f;
  }
#pragma unroll
  for (int n = 0; n < 2 * (r0 + 1); ++n) {
    const int j = n * 8 + t * 2;
    const float2 h = *reinterpret_cast<const float2*>(vec + kGhi * kC + j);
    const float2 l = *reinterpret_cast<const float2*>(vec + kGlo * kC + j);
    float2 s = make_float2(0.f, 0.f);
    if (RESETS) s = *reinterpret_cast<const float2*>(vec + kSeg * kC + j);
    float2 be = *reinterpret_cast<const float2*>(vec + kBeta * kC + j);
    mul2(be.x, be.y, f, f);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int rb = r < 2 ? r0 : r1, i = rb * 16 + g + 8 * (r & 1);
      if (n >= 2 * (rb + 1)) continue;
      const float* v = &x[(r < 2 ? 0 : 2 * (r0 + 1)) + n][2 * (r & 1)];
      const bool last = n >= 2 * rb;   // the diagonal block
      const bool n0 = (!RESETS || s.x == sg[r]) && (!last || (keys ? i > j : i >= j));
      const bool n1 = (!RESETS || s.y == sg[r]) && (!last || (keys ? i > j + 1 : i >= j + 1));
      float e0 = hi[r], e1 = hi[r], c0 = lo[r], c1 = lo[r];
      add2p(e0, e1, -h.x, -h.y);
      add2p(c0, c1, -l.x, -l.y);
      add2p(e0, e1, c0, c1);
      float y0 = ex2(n0 ? e0 : neg), y1 = ex2(n1 ? e1 : neg);
      mul2(y0, y1, be.x, be.y);
      mul2(y0, y1, v[0], v[1]);
      if (RESETS || last) {   // (a product that is not finite stays out of what it is not part of)
        y0 = n0 ? y0 : 0.f;
        y1 = n1 ? y1 : 0.f;
      }
      if (keys && last) {
        float* p = diag + rb * kDiag + (j - rb * 16) * 16 + i - rb * 16;
        p[0] = y0;
        p[16] = y1;
      } else {
        uint32_t m[2];
        split2<2>(y0, y1, m);
        unsigned char* p = planes + tile_at<64>(i, j >> 3) + (j & 7) * 2;
        *reinterpret_cast<uint32_t*>(p) = m[0];
        *reinterpret_cast<uint32_t*>(p + kTile) = m[1];
      }
    }
  }
}

// A bf16 tensor [batch, seqlen, rows, cols] as a map of boxes of 64 columns of one
// row of 64 tokens.
bool token_map(CUtensorMap* m, const void* base, int cols, int rows, int64_t L, int B, TokStride s,
               bool swizzle);

// After kParts: each segment's first state but the first's, into the slots of W.
cudaError_t launch_tc_join(const Args& a, cudaStream_t st);
// Of segments all at once the last one may write its state (to) where the first one
// still reads (*from): the first state is then taken from a copy.
cudaError_t copy_first(const Args& a, const float** from, const float* to, cudaStream_t st);
// Clears a.ctrl for a launch of `grid` CTAs.
cudaError_t start_work(const Args& a, int* grid, cudaStream_t st);

// A device's status word (after the stream's work), cleared if asked.  Each word is a
// copy and a wait of 10 us, which processes that never launched its kernels are spared.
template <typename W>
int read_status(W& word, const std::atomic<bool>& launched, int reset, cudaStream_t st, int* bits) {
  int h = 0;
  *bits = 0;
  if (!launched.load()) return 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&h, word, sizeof(int), 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && reset && h != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbolAsync(word, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  *bits = h;
  return (int)e;
}

int tc_prepare_status(int reset, cudaStream_t st, int* bits);
int tc_forward_status(int reset, cudaStream_t st, int* bits);
int tc_reverse_status(int reset, cudaStream_t st, int* bits);
int tc_grads_status(int reset, cudaStream_t st, int* bits);

// The chunks' vectors, T and P; then the chunks one after another.
cudaError_t launch_tc_prepare(const Args& a, cudaStream_t st);
cudaError_t launch_tc_forward(const Args& a, cudaStream_t st);
cudaError_t launch_tc_reverse(const Args& a, cudaStream_t st);
cudaError_t launch_tc_grads(const Args& a, cudaStream_t st);

}  // namespace delta
}  // namespace ssd
