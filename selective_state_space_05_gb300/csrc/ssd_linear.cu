// Projections of the block: out = act(x W^T + bias) + residual, and its
// backward dx = dpre W, dW = dpre^T x, dbias = sum dpre, dpre = dout act'(pre).
//
// All three products are one kernel, D[m,n] = sum_k A[m,k] B[n,k], on the
// tensor cores (tcgen05, accumulators in TMEM, operand tiles by TMA with the
// 128-byte swizzle).  An operand is read where it lies: K-major (x and W of
// the forward, dpre of dx) or MN-major (W of dx, dpre and x of dW), so nothing
// is transposed.
//
// fp32 runs on the same kernel: each operand is split beforehand into three
// bf16 planes hi + mid + lo, which hold its 24-bit significand exactly, and
// the six products down to 2^-24 (hi hi, hi mid, mid hi, mid mid, hi lo,
// lo hi) are more K steps of the same sum, the smallest first.  Infinities and
// NaN have no such planes: they are left out of them, and a launch that ends at
// once where there was none puts their products into the results.
//
// The kernel is persistent.  A pair of CTAs on two SMs walks output tiles of
// 256 x BN (cta_group::2: each SM reads half of B's tile, which the shared
// memory's bandwidth needs: with 128 x 256 tiles on one SM, 96 KB a K step are
// written and read in 512 tensor cycles, and it reached 1.5 PFLOP/s); small
// products take 128 x BN tiles on single CTAs.  In a CTA one
// thread issues the TMA loads, one the MMAs, and eight warps take finished
// accumulators out of TMEM (two, so that the next MMAs run meanwhile) into
// registers, turn them through shared memory so that rows are written in whole
// sectors, and apply bias, activation and residual on the way.  Tiles that would
// fill the SMs only partly are split along K over them: each split writes its
// partial sums in fp32 and a second kernel adds them in a fixed order and applies
// the same epilogue.
//
// A few rows (decoding) are bound by the weight's bytes: the skinny kernels
// stream W through registers once, all of its loads in flight, with mma.sync for
// bf16 (the weight's rows are the MMA's 16 rows, the tokens its 8 columns) and
// fp32 FMAs for fp32 (once for every 8 rows).
//
// Measured on one GB300 (bf16, of 1885 TFLOP/s for a library product):
// 32768 x 2560 -> 10576 forward 915-943 us (1.94-1.88 PFLOP/s, the tensor pipe 93 %
// active in a capture), dx 923-943 us, dW 997-1054 us; 1021 x 5120 -> 2560 into an fp32
// residual 35 us, where 64 of 76 pairs hold one tile each and its last epilogue
// has nothing to hide behind; 8 x 2560 -> 10576 10.3 us (5.3 TB/s of weight).
// fp32, 4095 x 2048 -> 4384: forward 282 us, dx 306, dW 292 with the splitting
// into planes (six bf16 products: 1.57, 1.44 and 1.51 PFLOP/s of them).
#include <cudaTypedefs.h>
#include <cuda_fp16.h>
#include <stdio.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "../../include/ssd_block.h"
#include "ssd_common.cuh"
#include "ssd_row.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace linear {

constexpr int kBM = 128, kBK = 64;
constexpr int kEpiWarps = 8;              // two a quarter of the TMEM lanes: every other 32 columns
constexpr int kThreads = 64 + 32 * kEpiWarps;   // warp 0: TMA, 1: MMA, then the epilogue
// K steps that one TMEM accumulator takes where the result is kept in fp32.
// The tensor core's fp32 sum rounds towards zero at every MMA, an error that
// grows with their number (relative 3.9e-6 after 320 MMAs, K = 5120, measured);
// short sums are added up in registers, to nearest, instead.  Relative error of the
// whole result at K = 512 to 10576, where fp32 FMAs reach 4e-7 to 1.8e-6:
// fp32 operands 4.8e-7 with 8 steps (16: 1.0e-6); the small products of planes,
// which come first, add nothing to it and take long sums, which also lets the MMAs
// run on while the epilogue is busy with the tile before (4095 x 2048 -> 4384 with
// bias: 304 us; 16 steps throughout 323, 8 throughout 341).  bf16 operands 1.0e-6
// with 16 steps (8: 4.8e-7, but 8192 x 1024 -> 2560 into a residual 115 us instead
// of 95).
constexpr int kExactSteps = 16, kPlanesSteps = 8, kLeadSteps = 64;
// Where it is rounded to bf16 afterwards an accumulator takes more: an MMA loses
// less than 2^-23 of the running sum, which for terms of one sign is half of the
// total on average, so 1024 MMAs lose at most 2^-14, a 32nd of the least half step
// of bf16.  (Summed in one accumulator, a dW over 2^24 tokens of one sign was
// 0.8 % short.)
constexpr int kBf16Steps = 256;
constexpr unsigned long long kWaitNs = 2000000000ull;   // limit of any single wait: 2 s
constexpr uint32_t kSleepNs = 20000;

// Sticky status of this device: nonzero once a wait gave up (ssd_scan_status).
__device__ int g_status_linear;

// (of bf16 data: with the exponentials that are exact enough for it, row::sigmoid)
enum { kActNone = 0, kActSilu = 1, kActGelu = 2, kActSiluBf16 = 3, kActGeluBf16 = 4 };
int act_of(ssd_activation_t a, ssd_dtype_t dtype) {
  return a == SSD_ACT_NONE || dtype == SSD_DTYPE_F32 ? (int)a : (int)a + 2;
}
enum { kNone = 0, kF32 = 1, kBf16 = 2, kF16 = 3 };

// What happens to a sum on its way out: out = act(sum + bias) + res, and pre =
// sum + bias where the backward will want it.
struct Epilogue {
  const void* bias;
  const void* res;
  void* out;
  void* pre;
  int64_t res_ld, out_ld;
  uint8_t bias_t, res_t, out_t, pre_t, act;
  bool wide;    // four columns at once: every row of every tensor stays aligned for it
  bool wide8;   // eight
};

__device__ __forceinline__ float act_f(int act, float v) {
  if (act == kActSilu) return v * row::sigmoid<float>(v);
  if (act == kActSiluBf16) return v * row::sigmoid<__nv_bfloat16>(v);
  if (act != kActNone) return 0.5f * v * (1.f + erff(v * 0.70710678f));
  return v;
}
__device__ __forceinline__ float dact_f(int act, float v) {
  if (act == kActSilu || act == kActSiluBf16) {
    const float s = act == kActSilu ? row::sigmoid<float>(v) : row::sigmoid<__nv_bfloat16>(v);
    return s * (1.f + v * (1.f - s));
  }
  if (act != kActNone) {
    const float q = -0.5f * v * v;
    return 0.5f * (1.f + erff(v * 0.70710678f)) +
           v * 0.39894228f * (act == kActGelu ? expf(q) : __expf(q));
  }
  return 1.f;
}

// The half that pre is kept in: beyond its range act' is flat, so the largest
// half stands for it (an infinity would make silu' a NaN).
__device__ __forceinline__ float half_range(float v) {
  return v > 65504.f ? 65504.f : v < -65504.f ? -65504.f : v;   // NaN stays
}

__device__ __forceinline__ float get1(const void* p, int t, int64_t i) {
  if (t == kF32) return static_cast<const float*>(p)[i];
  if (t == kF16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void put1(void* p, int t, int64_t i, float v) {
  if (t == kF32) static_cast<float*>(p)[i] = v;
  else if (t == kF16) static_cast<__half*>(p)[i] = __float2half_rn(half_range(v));
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ void get4(const void* p, int t, int64_t i, float (&v)[4]) {
  if (t == kF32) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + i);
    v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xFFFF0000u);
    v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void put4(void* p, int t, int64_t i, const float (&v)[4]) {
  if (t == kF32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
  } else if (t == kF16) {
    const __half2 a = __floats2half2_rn(half_range(v[0]), half_range(v[1]));
    const __half2 b = __floats2half2_rn(half_range(v[2]), half_range(v[3]));
    *reinterpret_cast<uint2*>(static_cast<__half*>(p) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + i) =
        make_uint2(tc::pack_bf16x2(v[0], v[1]), tc::pack_bf16x2(v[2], v[3]));
  }
}

// The residual at row m, columns n .. n + 3 (zeros past N, and without one).
// Apart from finish4, so that a thread has all of its loads in flight before
// its first store (the output may be the residual's memory).
__device__ __forceinline__ void residual4(const Epilogue& e, int64_t m, int64_t n, int64_t N,
                                          float (&r)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = 0.f;
  if (!e.res) return;
  if (e.wide) {
    if (n < N) get4(e.res, e.res_t, m * e.res_ld + n, r);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) r[i] = get1(e.res, e.res_t, m * e.res_ld + n + i);
  }
}

// Sums of row m, columns n .. n + 3 (those below N).  v is finished in place.
__device__ __forceinline__ void finish4(const Epilogue& e, int64_t m, int64_t n, int64_t N,
                                        float (&v)[4], const float (&res)[4]) {
  if (e.wide) {
    if (n >= N) return;
    if (e.bias) {
      float b[4];
      get4(e.bias, e.bias_t, n, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += b[i];
    }
    if (e.pre) put4(e.pre, e.pre_t, m * N + n, v);
    if (e.act != kActNone) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = act_f(e.act, v[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e.res) v[i] += res[i];
    put4(e.out, e.out_t, m * e.out_ld + n, v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n + i >= N) return;
      float s = v[i] + (e.bias ? get1(e.bias, e.bias_t, n + i) : 0.f);
      if (e.pre) put1(e.pre, e.pre_t, m * N + n + i, s);
      s = act_f(e.act, s);
      if (e.res) s += res[i];
      put1(e.out, e.out_t, m * e.out_ld + n + i, s);
    }
  }
}

// Eight consecutive elements (16-byte accesses).
__device__ __forceinline__ void get8(const void* p, int t, float (&v)[8]) {
  if (t == kF32) {
    const float4 a = static_cast<const float4*>(p)[0], b = static_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else if (t == kF16) {
    const uint4 w = *static_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
    row::unpack(*static_cast<const uint4*>(p), v);
  }
}
__device__ __forceinline__ void put8(void* p, int t, const float (&v)[8]) {
  if (t == kF32) {
    static_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    static_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (t == kF16) {
        const __half2 h = __floats2half2_rn(half_range(v[2 * i]), half_range(v[2 * i + 1]));
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        u[i] = tc::pack_bf16x2(v[2 * i], v[2 * i + 1]);
      }
    }
    *static_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// v[r] to element at + r * ld of p, r < rows.
__device__ __forceinline__ void put_column(void* p, int t, int64_t at, int64_t ld, int rows,
                                           const float (&v)[8]) {
#pragma unroll
  for (int r = 0; r < 8; ++r)
    if (r < rows) put1(p, t, at + r * ld, v[r]);
}

// Columns col .. col + 7 of a row whose tensors are aligned for eight columns
// (whole) or for four; more: whether the second four are below N.
__device__ __forceinline__ void get8(const void* p, int t, bool whole, bool more, float (&v)[8]) {
  if (whole) {
    get8(p, t, v);
    return;
  }
  float a[4], b[4] = {0.f, 0.f, 0.f, 0.f};
  get4(p, t, 0, a);
  if (more) get4(p, t, 4, b);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = a[j];
    v[4 + j] = b[j];
  }
}
__device__ __forceinline__ void put8(void* p, int t, bool whole, bool more, const float (&v)[8]) {
  if (whole) {
    put8(p, t, v);
    return;
  }
  const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
  put4(p, t, 0, a);
  if (more) put4(p, t, 4, b);
}

// ------------------------------------------------------------------ the product

struct Gemm {
  int64_t M, N;
  int kblocks;        // K in steps of kBK
  int pairs;          // products of planes: 1, or 6 for fp32
  int tiles_m, tiles_n;
  int full;           // tiles [0, full) are computed whole, the others ("the tail") in
  int splits, steps_per_split;   // splits of K each, joined afterwards where splits > 1
  int bn;             // tile width, a multiple of 32 up to 256
  int stages;         // operand tiles in flight
  int group_m;        // tiles of M walked together (L2 reuse)
  int run;            // K steps an accumulator takes before it is added to the registers',
  int lead;           // except for the first `lead` steps, the small products of planes:
  float* partial;     // [tail tile][splits][rows of a tile][bn] where splits > 1
  Epilogue e;
};

// The planes of the q-th product of an fp32 sum, smallest first.
__device__ __forceinline__ void planes_of(int pairs, int q, int& a, int& b) {
  if (pairs == 1) {
    a = b = 0;
    return;
  }
  switch (q) {
    case 0: a = 0; b = 2; break;
    case 1: a = 2; b = 0; break;
    case 2: a = 1; b = 1; break;
    case 3: a = 0; b = 1; break;
    case 4: a = 1; b = 0; break;
    default: a = 0; b = 0; break;
  }
}

// CG CTAs work on a tile of CG * kBM x BN: a CTA holds kBM rows of A and BN / CG
// rows of B (whole blocks of 64 where B is MN-major).
constexpr int kStageA = kBM * kBK * 2;
constexpr int kOperandBytes = 192 * 1024, kMaxStages = 10;
__host__ __device__ constexpr int rows_b(int cg, int bn, bool mn) {
  return mn ? (bn / cg + 63) / 64 * 64 : bn / cg;
}
__host__ __device__ constexpr int stage_b(int cg, int bn, bool mn) {
  return rows_b(cg, bn, mn) * kBK * 2;
}
constexpr uint32_t kTmemCols = 512;   // two accumulators of up to 256 columns

struct alignas(1024) Smem {
  unsigned char operands[kOperandBytes];   // stages of A's tile, then B's
  float turn[kEpiWarps][32 * 32];
  uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2], drain;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "shared memory");

__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// Waits for a phase; gives up after kWaitNs, or soon after another role of the
// CTA gave up.  Returns whether the phase completed.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, int* abort) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = now_ns();
  for (;;) {
    if (tc::mbar_try_wait_sleep(bar, parity, kSleepNs)) return true;
    if (*reinterpret_cast<volatile int*>(abort)) return false;
    if (now_ns() - t0 > kWaitNs) {
      *reinterpret_cast<volatile int*>(abort) = 1;
      atomicOr(&g_status_linear, 1);
      return false;
    }
  }
}
// For work of its own that is still in flight at the end: not cut short by an abort.
__device__ __forceinline__ void wait_drain(uint64_t* bar, uint32_t parity) {
  const unsigned long long t0 = now_ns();
  while (!tc::mbar_try_wait_sleep(bar, parity, kSleepNs))
    if (now_ns() - t0 > kWaitNs) {
      atomicOr(&g_status_linear, 2);
      return;
    }
}

// One stage's tile of an operand: `rows` (at most MOST) rows of M or N from r0,
// kBK of K from k0.  bar: the barrier, for a CTA pair as a shared::cluster
// address.
template <int CG, int MOST, bool MN>
__device__ __forceinline__ void load_tile(unsigned char* dst, const CUtensorMap* map, uint64_t* bar,
                                          uint32_t pair_bar, int rows, int r0, int k0, int plane) {
#pragma unroll
  for (int j = 0; j < (MN ? MOST / 64 : 1); ++j) {
    if (MN && 64 * j >= rows) break;
    unsigned char* to = dst + j * (kBK * 128);
    const int x = MN ? r0 + 64 * j : k0, y = MN ? k0 : r0;
    if constexpr (CG == 2) tc::tma_load_3d_pair(to, map, pair_bar, x, y, plane);
    else tc::tma_load_3d(to, map, bar, x, y, plane);
  }
}
template <bool MN>
__device__ __forceinline__ uint64_t tile_desc(const unsigned char* p) {
  return MN ? tc::sdesc_sw128(tc::smem_u32(p), kBK * 128, 1024)
            : tc::sdesc_sw128(tc::smem_u32(p), 16, 1024);
}

// Tile number -> its place.  Tiles run down group_m rows of tiles before the
// next column, so that the CTAs at work at one time share operands in L2.
__host__ __device__ __forceinline__ void place_of(const Gemm& p, int t, int& tm, int& tn) {
  const int per = p.group_m * p.tiles_n;
  const int g = t / per, r = t - g * per;
  const int left = p.tiles_m - g * p.group_m, gm = left < p.group_m ? left : p.group_m;
  tm = g * p.group_m + r % gm;
  tn = r / gm;
}

// A work item: a whole tile, or one split of a tail tile; the K steps [k0, k1).
struct Item {
  int tm, tn, k0, k1;
  int part;   // of the tail: its place in `partial`; -1: finished here
};
__device__ __forceinline__ Item item_of(const Gemm& p, int item, int all_steps) {
  Item w;
  w.k0 = 0;
  w.k1 = all_steps;
  w.part = -1;
  int t = item;
  if (item >= p.full && p.splits > 1) {
    const int j = item - p.full, q = j / p.splits, split = j - q * p.splits;
    t = p.full + q;
    w.part = j;
    w.k0 = split * p.steps_per_split;
    w.k1 = min(w.k0 + p.steps_per_split, all_steps);
  }
  place_of(p, t, w.tm, w.tn);
  return w;
}

// Where the run of K steps ends that begins at r0, of an item that ends at k1.
__device__ __forceinline__ int run_end(const Gemm& p, int r0, int k1) {
  return min(r0 < p.lead ? min(r0 + kLeadSteps, p.lead) : r0 + p.run, k1);
}

// A CTA pair (CG 2): each CTA loads its own operand rows, counted on the
// leader's `full`; the leader issues the MMAs and signals `empty` and `tfull`
// of both; both CTAs' epilogues arrive on the leader's `tempty`.
// EXACT: sums in runs of p.run K steps (fp32 results, long sums); PLAIN: no bias,
// pre, activation or residual.  Apart, because one kernel with all of it was 150 KB
// of code and spilled.
template <int CG, bool AMN, bool BMN, bool EXACT, bool PLAIN>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(CG, 1, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                const __grid_constant__ Gemm p) {
  extern __shared__ unsigned char raw[];
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int S = p.stages, BN = p.bn;
  const int rowsB = rows_b(CG, BN, BMN), stage = kStageA + rowsB * kBK * 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? (int)tc::cluster_rank() : 0;
  const int first = blockIdx.x / CG, stride = gridDim.x / CG;
  const int items = p.full + (p.tiles_m * p.tiles_n - p.full) * p.splits;
  const int all_steps = p.kblocks * p.pairs;

  if (warp == 0 && lane == 0) {
    for (int i = 0; i < S; ++i) {
      tc::mbar_init(&s.full[i], 1);
      tc::mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s.tfull[i], 1);
      tc::mbar_init(&s.tempty[i], CG * kEpiWarps);
    }
    tc::mbar_init(&s.drain, 1);
    tc::mbar_fence_init();
    s.abort = 0;
    tc::tma_prefetch_desc(&ma);
    tc::tma_prefetch_desc(&mb);
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      tc::tmem_alloc_pair(&s.tmem, kTmemCols);
      tc::tmem_relinquish_pair();
    } else {
      tc::tmem_alloc(&s.tmem, kTmemCols);
      tc::tmem_relinquish();
    }
    tc::fence_before_sync();
  }
  __syncthreads();
  if constexpr (CG == 2) tc::cluster_sync();   // the peer's barriers are ready
  tc::fence_after_sync();
  const uint32_t tmem = s.tmem;

  // The TMA and MMA warps run their loops converged, one elected lane issuing:
  // descriptors and coordinates then live in uniform registers.  (With the
  // loops inside one lane's branch, a K step's four MMAs and their commit took
  // about 500 cycles to issue, as long as the MMAs themselves.)
  if (warp == 0) {
    int st = 0;
    uint32_t ph = 0;
    int issued = 0;
    bool ok = true;
    for (int it = first; it < items && ok; it += stride) {
      const Item w = item_of(p, it, all_steps);
      const int tm = w.tm, tn = w.tn, k0 = w.k0, k1 = w.k1;
      int q = k0 / p.kblocks, kb = k0 - q * p.kblocks;   // product of planes, K step in it
      int pa, pb;
      planes_of(p.pairs, q, pa, pb);
      for (int k = k0; k < k1; ++k) {
        if (kb == p.kblocks) {
          kb = 0;
          planes_of(p.pairs, ++q, pa, pb);
        }
        const int kk = kb++ * kBK;
        ok = __all_sync(0xffffffffu, wait_phase(&s.empty[st], ph ^ 1, &s.abort));
        if (!ok) break;
        if (tc::elect_one()) {
          if (rank == 0)
            tc::mbar_arrive_expect_tx(&s.full[st], CG * stage);
          const uint32_t bar = CG == 2 ? tc::mapa(&s.full[st], 0) : 0;
          unsigned char* at = s.operands + st * stage;
          load_tile<CG, kBM, AMN>(at, &ma, &s.full[st], bar, kBM, (tm * CG + rank) * kBM, kk, pa);
          load_tile<CG, 256 / CG, BMN>(at + kStageA, &mb, &s.full[st], bar, rowsB,
                             tn * BN + rank * (BN / CG), kk, pb);
        }
        __syncwarp();
        ++issued;
        if (++st == S) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    // no copy outlives the CTA (a pair's are counted by the leader, which
    // both CTAs wait for at the end)
    if (!ok && rank == 0) {
      for (int i = max(0, issued - S); i < issued; ++i)
        wait_drain(&s.full[i % S], (i / S) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t idesc = tc::idesc_bf16(CG * kBM, BN, AMN, BMN);
      auto commit = [](uint64_t* bar) {
        if (tc::elect_one()) {
          if constexpr (CG == 2) tc::mma_commit_pair(bar);
          else tc::mma_commit(bar);
        }
        __syncwarp();
      };
      const uint64_t da0 = tile_desc<AMN>(s.operands), db0 = tile_desc<BMN>(s.operands + kStageA);
      int st = 0, n = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int it = first; it < items && ok; it += stride) {
        const Item w = item_of(p, it, all_steps);
        const int k0 = w.k0, k1 = w.k1;
        for (int r0 = k0, r1; r0 < k1 && ok; r0 = r1, ++n) {
          r1 = EXACT ? run_end(p, r0, k1) : k1;
          const int buf = n & 1;
          ok = __all_sync(0xffffffffu,
                          wait_phase(&s.tempty[buf], ((n >> 1) & 1) ^ 1, &s.abort));
          tc::fence_after_sync();
          for (int k = r0; k < r1 && ok; ++k) {
            ok = __all_sync(0xffffffffu, wait_phase(&s.full[st], ph, &s.abort));
            if (!ok) break;
            tc::fence_after_sync();
            // (descriptors count 16-byte units)
            const uint64_t da = da0 + st * (stage >> 4), db = db0 + st * (stage >> 4);
            if (tc::elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kBK / 16; ++kk) {
                const uint64_t a = da + kk * (AMN ? 128 : 2), b = db + kk * (BMN ? 128 : 2);
                if constexpr (CG == 2)
                  tc::mma_ss_pair(tmem + buf * 256, a, b, idesc, k > r0 || kk > 0);
                else
                  tc::mma_ss(tmem + buf * 256, a, b, idesc, k > r0 || kk > 0);
              }
            }
            __syncwarp();
            commit(&s.empty[st]);
            if (++st == S) {
              st = 0;
              ph ^= 1;
            }
          }
          if (ok) commit(&s.tfull[buf]);
        }
      }
      // every MMA has finished before the operands' memory and TMEM are given back
      commit(&s.drain);
      wait_drain(&s.drain, 0);
      __syncwarp();
    }
  } else {
    // a quarter of the TMEM lanes and every other 32 columns
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    float* turn = s.turn[warp - 2];
    int n = 0;
    bool ok = true;
    for (int it = first; it < items; it += stride) {
      const Item w = item_of(p, it, all_steps);
      const int tm = w.tm, tn = w.tn, k0 = w.k0, k1 = w.k1;
      const bool parts = w.part >= 0;
      auto filled = [&](int i) {   // one verdict for the warp: TMEM loads take all of its lanes
        const bool r =
            __all_sync(0xffffffffu, wait_phase(&s.tfull[i & 1], (i >> 1) & 1, &s.abort));
        tc::fence_after_sync();
        return r;
      };
      auto release = [&](int i) {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2) tc::mbar_arrive_cluster(tc::mapa(&s.tempty[i & 1], 0));
          else tc::mbar_arrive(&s.tempty[i & 1]);
        }
      };
      const bool has_res = !PLAIN && p.e.res && !parts;
      if (has_res) {
        // the residual on its way to L2 while the sums are made: a row a lane
        const int64_t m = ((int64_t)tm * CG + rank) * kBM + q * 32 + lane;
        if (m < p.M)
          for (int c = half * 32; c < BN; c += 64) {
            const int64_t n = (int64_t)tn * BN + c;
            if (n < p.N)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(
                  static_cast<const char*>(p.e.res) +
                  (m * p.e.res_ld + n) * (p.e.res_t == kF32 ? 4 : 2)));
          }
      }
      if (EXACT && run_end(p, k0, k1) < k1) {
        // the runs' sums in registers; their total goes back to the last run's
        // place in TMEM
        float acc[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[c][i] = 0.f;
        for (int r0 = k0, r1; r0 < k1; r0 = r1, ++n) {
          r1 = run_end(p, r0, k1);
          ok = filled(n);
          if (!ok) break;
          const uint32_t at = tmem + (n & 1) * 256 + lanes;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int col = (2 * c + half) * 32;
            if (col < BN) {
              uint32_t r[32];
              tc::tmem_ld32(at + col, r);
              tc::tmem_ld_wait_regs(r);
#pragma unroll
              for (int i = 0; i < 32; ++i) acc[c][i] += __uint_as_float(r[i]);
            }
          }
          if (r1 < k1) release(n);
        }
        if (!ok) break;
        --n;
        const uint32_t at = tmem + (n & 1) * 256 + lanes;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int col = (2 * c + half) * 32;
          if (col < BN) {
            uint32_t r[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(acc[c][i]);
            tc::tmem_st32(at + col, r);
          }
        }
        tc::tmem_st_wait();
      } else {
        ok = filled(n);
        if (!ok) break;
      }
      // Rows by lane become eight rows of four lanes at a time, eight columns a
      // lane.  The 16-byte pieces of a row are exchanged by its number, so that
      // both directions reach all banks.
      const uint32_t at = tmem + (n & 1) * 256 + lanes;
      const int64_t m0 = ((int64_t)tm * CG + rank) * kBM + q * 32;
      const int64_t n0 = (int64_t)tn * BN;
      const int rows = parts ? 32 : (int)min((int64_t)32, p.M - m0);   // <= 0: none of this warp's
      const int rr = lane >> 2, cc = lane & 3;
      const int out_t = parts ? kF32 : p.e.out_t;
      const int64_t out_ld = parts ? BN : p.e.out_ld;
      const int oe = out_t == kF32 ? 4 : 2;
      // this lane's place in the tile's first row and column block
      char* const base =
          parts ? reinterpret_cast<char*>(
                      p.partial + (((int64_t)w.part * CG + rank) * kBM + q * 32 + rr) * BN + 8 * cc)
                : static_cast<char*>(p.e.out) + ((m0 + rr) * out_ld + n0 + 8 * cc) * oe;
      const bool whole = parts || p.e.wide8, wide = whole || p.e.wide;
      const bool plain = PLAIN || parts;
#pragma unroll 1
      for (int c = half * 32; c < BN; c += 64) {
        const int64_t col = n0 + c + 8 * cc;
        const bool in = wide && (parts || col < p.N), more = parts || col + 4 < p.N;
        // the residual first: its loads are in flight during the TMEM load, all
        // of them before the first store
        float res[4][8];
        if (in && has_res) {
          const int re = p.e.res_t == kF32 ? 4 : 2;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (8 * i + rr < rows)
              get8(static_cast<const char*>(p.e.res) + ((m0 + 8 * i + rr) * p.e.res_ld + col) * re,
                   p.e.res_t, whole, more, res[i]);
        }
        uint32_t r[32];
        __syncwarp();
        tc::tmem_ld32(at + c, r);
        tc::tmem_ld_wait_regs(r);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(turn + lane * 32 + 4 * (i ^ (lane & 7))) =
              make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        __syncwarp();
        auto sums = [&](int r, float (&v)[8]) {
          const float4 x = *reinterpret_cast<const float4*>(turn + r * 32 + 4 * ((2 * cc) ^ (r & 7)));
          const float4 y =
              *reinterpret_cast<const float4*>(turn + r * 32 + 4 * ((2 * cc + 1) ^ (r & 7)));
          v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
          v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
        };
        if (in) {
          char* o = base + c * oe;
          const int64_t step = 8 * out_ld * oe;
          if (plain) {   // all of the sums read, then all stored
            float v[4][8];
#pragma unroll
            for (int i = 0; i < 4; ++i) sums(8 * i + rr, v[i]);
            if (out_t == kF32) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (8 * i + rr < rows) put8(o + i * step, kF32, whole, more, v[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (8 * i + rr < rows) put8(o + i * step, kBf16, whole, more, v[i]);
            }
          } else {
            float bias[8];
            if (p.e.bias)
              get8(static_cast<const char*>(p.e.bias) + col * (p.e.bias_t == kF32 ? 4 : 2),
                   p.e.bias_t, whole, more, bias);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (8 * i + rr < rows) {
                float v[8];
                sums(8 * i + rr, v);
                if (p.e.bias) {
#pragma unroll
                  for (int j = 0; j < 8; ++j) v[j] += bias[j];
                }
                if (p.e.pre)
                  put8(static_cast<char*>(p.e.pre) +
                           ((m0 + 8 * i + rr) * p.N + col) * (p.e.pre_t == kF32 ? 4 : 2),
                       p.e.pre_t, whole, more, v);
                if (p.e.act != kActNone) {
#pragma unroll
                  for (int j = 0; j < 8; ++j) v[j] = act_f(p.e.act, v[j]);
                }
                if (has_res) {
#pragma unroll
                  for (int j = 0; j < 8; ++j) v[j] += res[i][j];
                }
                put8(o + i * step, out_t, whole, more, v);
              }
            }
          }
        } else if (!wide) {   // a column a lane, eight rows at a time
          const int64_t cl = n0 + c + lane;
          if (cl < p.N) {
            const float b = !PLAIN && p.e.bias ? get1(p.e.bias, p.e.bias_t, cl) : 0.f;
#pragma unroll 1
            for (int r0 = 0; r0 < rows; r0 += 8) {
              float v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int r = r0 + i;
                v[i] = turn[r * 32 + 4 * ((lane >> 2) ^ (r & 7)) + (lane & 3)] + b;
              }
              const int left = rows - r0;
              if constexpr (!PLAIN) {
                if (p.e.pre)
                  put_column(p.e.pre, p.e.pre_t, (m0 + r0) * p.N + cl, p.N, left, v);
                if (p.e.act != kActNone) {
#pragma unroll
                  for (int i = 0; i < 8; ++i) v[i] = act_f(p.e.act, v[i]);
                }
                if (has_res) {
                  float res[8];
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    res[i] =
                        i < left ? get1(p.e.res, p.e.res_t, (m0 + r0 + i) * p.e.res_ld + cl) : 0.f;
#pragma unroll
                  for (int i = 0; i < 8; ++i) v[i] += res[i];
                }
              }
              put_column(p.e.out, out_t, (m0 + r0) * out_ld + cl, out_ld, left, v);
            }
          }
        }
      }
      release(n);
      ++n;
    }
  }
  __syncthreads();
  if (CG == 2 && rank == 1 && warp == 1) {
    // the leader's commits arrive at the peer's barriers too: its memory stays
    // until the last of them has.  This CTA's other warps are done, so its last
    // tile is: what is left of the leader's work is short, and so is the wait,
    // however long the launch was.
    wait_drain(&s.drain, 0);
    __syncwarp();
  }
  tc::fence_after_sync();
  if constexpr (CG == 2) {
    tc::cluster_sync();   // nothing of the peer's is needed or written any more
    if (warp == 1) tc::tmem_dealloc_pair(tmem, kTmemCols);
  } else {
    if (warp == 1) tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// Adds the partial sums of the tail's tiles, in order, and finishes them: four
// columns a thread, a tile a blockIdx.y.
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Gemm p, int rows) {
  const int i = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= rows * p.bn) return;
  const int r = i / p.bn, c = i - r * p.bn;
  int tm, tn;
  place_of(p, p.full + blockIdx.y, tm, tn);
  const int64_t m = (int64_t)tm * rows + r, n = (int64_t)tn * p.bn + c;
  if (m >= p.M || n >= p.N) return;
  float v[4] = {0.f, 0.f, 0.f, 0.f}, res[4];
  residual4(p.e, m, n, p.N, res);
  const float* part = p.partial + (int64_t)blockIdx.y * p.splits * rows * p.bn + i;
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) {
    const float4 f = *reinterpret_cast<const float4*>(part + (int64_t)s * rows * p.bn);
    v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
  }
  finish4(p.e, m, n, p.N, v, res);
}

// ------------------------------------------------------- operands made ready

// src (times act'(pre)) as bf16 planes [planes][R][ld] (planes 0: none), and
// its column sums over this CTA's rows (colsum: [gridDim.y][C], or null).
// Three planes hold a finite fp32 value exactly (above 2^-110, whose third
// plane is still normal): each takes the next 8 bits of its significand,
// rounded, the next one the remainder; where rounding would overflow, 8 bits
// towards zero each (24 in all: exact as well).
// Infinities and NaN get zeros, and flags tell which CTAs met one.
struct Prep {
  const void* src;
  const void* pre;
  __nv_bfloat16* out;
  float* colsum;
  int* flags;   // of three planes: [gridDim.y][gridDim.x]
  int64_t R, src_ld, ld, rows_per;
  int C;
  uint8_t src_t, pre_t, act, planes;
};
// Eight consecutive elements from an address that is aligned to its element
// only: the aligned 16-byte words that hold them (none past `end`, the end of
// the row, is touched), moved down by the offset in steps of 2, 1 and 1/2 words.
__device__ __forceinline__ void get8_any(const void* p, int t, const void* end, float (&v)[8]) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), base = a & ~(uintptr_t)15;
  const uint4* q = reinterpret_cast<const uint4*>(base);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int off = (int)(a & 15) >> 2, n = t == kF32 ? 3 : 2;   // in words; 16-byte words needed
  uint32_t u[12];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint4 w =
        i < n && reinterpret_cast<uintptr_t>(q + i) < reinterpret_cast<uintptr_t>(end) ? q[i] : zero;
    u[4 * i] = w.x; u[4 * i + 1] = w.y; u[4 * i + 2] = w.z; u[4 * i + 3] = w.w;
  }
  if (off & 2) {
#pragma unroll
    for (int i = 0; i < 10; ++i) u[i] = u[i + 2];
  }
  if (off & 1) {
#pragma unroll
    for (int i = 0; i < 9; ++i) u[i] = u[i + 1];
  }
  if (t == kF32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
    return;
  }
  if (a & 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __funnelshift_r(u[i], u[i + 1], 16);
  }
  if (t == kF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
    row::unpack(make_uint4(u[0], u[1], u[2], u[3]), v);
  }
}

// Whether one of eight packed bf16 is an infinity or a NaN.
__device__ __forceinline__ bool beyond(const uint32_t (&u)[4]) {
  uint32_t most = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) most = __vmaxu2(most, u[j] & 0x7FFF7FFFu);
  return (most & 0xFFFFu) >= 0x7F80u || most >= 0x7F800000u;
}

// Eight consecutive columns a thread; ANY: rows of any alignment and length; SPLIT:
// three planes.
template <bool ANY, bool SPLIT>
__global__ void __launch_bounds__(128) prep_kernel(const __grid_constant__ Prep p) {
  const int c = (blockIdx.x * 128 + threadIdx.x) * 8;
  const int64_t r0 = (int64_t)blockIdx.y * p.rows_per;
  const int64_t r1 = c < p.C ? min(r0 + p.rows_per, p.R) : r0;   // past the row: nothing
  bool far = false;   // a value that has no first plane
  const int se = p.src_t == kF32 ? 4 : 2, pe = p.pre_t == kF32 ? 4 : 2;
  const int left = p.C - c;
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.f;
  // kAhead rows' loads before the first store (which may not be moved over loads)
  constexpr int kAhead = 4;
  for (int64_t rb = r0; rb < r1; rb += kAhead) {
    float v[kAhead][8], q[kAhead][8];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t r = min(rb + i, r1 - 1);
      const char* src = static_cast<const char*>(p.src) + (r * p.src_ld + c) * se;
      if (ANY) get8_any(src, p.src_t, src + (int64_t)left * se, v[i]);
      else get8(src, p.src_t, v[i]);
    }
    if (p.pre) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t r = min(rb + i, r1 - 1);
        const char* pre = static_cast<const char*>(p.pre) + (r * p.C + c) * pe;
        if (ANY) get8_any(pre, p.pre_t, pre + (int64_t)left * pe, q[i]);
        else get8(pre, p.pre_t, q[i]);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= dact_f(p.act, q[i][j]);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (rb + i >= r1) break;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += v[i][j];
      if (!SPLIT && p.planes == 0) continue;
      __nv_bfloat16* o = p.out + (rb + i) * p.ld + c;   // (ld is a multiple of 8: the pad may be written)
      uint32_t u[4];
#pragma unroll
      for (int k = 0; k < (SPLIT ? 3 : 1); ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = tc::pack_bf16x2(v[i][2 * j], v[i][2 * j + 1]);
        if (SPLIT && k == 0) far |= beyond(u);
        if (SPLIT && k < 2) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[i][2 * j] -= __uint_as_float(u[j] << 16);
            v[i][2 * j + 1] -= __uint_as_float(u[j] & 0xFFFF0000u);
          }
        }
        *reinterpret_cast<uint4*>(o + k * p.R * p.ld) = make_uint4(u[0], u[1], u[2], u[3]);
      }
    }
  }
  bool met = false;   // an infinity or NaN
  if (SPLIT && far) {   // the thread's part once more, value by value
    for (int64_t r = r0; r < r1; ++r) {
#pragma unroll 1
      for (int j = 0; j < min(8, left); ++j) {
        float v = static_cast<const float*>(p.src)[r * p.src_ld + c + j];
        if (p.pre) v *= dact_f(p.act, static_cast<const float*>(p.pre)[r * p.C + c + j]);
        if (!isfinite(v)) {
          v = 0.f;
          met = true;
        }
        // towards zero where rounding would overflow: no sum of the planes is
        // beyond the value
        const bool chop = fabsf(v) >= 0x1.FFp127f;
        for (int k = 0; k < 3; ++k) {
          const __nv_bfloat16 h = chop ? __float2bfloat16_rz(v) : __float2bfloat16_rn(v);
          p.out[(k * p.R + r) * p.ld + c + j] = h;
          v -= __bfloat162float(h);
        }
      }
    }
  }
  if (p.colsum) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) p.colsum[(int64_t)blockIdx.y * p.C + c + j] = sum[j];
  }
  if (p.flags) {
    met = __syncthreads_or(met);
    if (threadIdx.x == 0) p.flags[blockIdx.y * gridDim.x + blockIdx.x] = met;
  }
}

// A side of an fp32 product D[m,n] = sum_k A[m,k] B[n,k] as it was given: element
// (r, k) is src[r * ld + k], or src[k * ld + r] (mn), times act'(pre) of the same
// place (rows of pre are pre_ld apart).  flags: of prep_kernel's blocks, flags_y of
// rows_per rows by flags_x of 1024 columns of src, which hold infinities or NaN.
struct Given {
  const float* src;
  const float* pre;
  const int* flags;
  int64_t ld, pre_ld, rows_per;
  int flags_x, flags_y;
  uint8_t act;
  bool mn;
  __device__ __forceinline__ float at(int64_t r, int64_t k) const {
    const float v = src[mn ? k * ld + r : r * ld + k];
    return pre ? v * dact_f(act, pre[mn ? k * pre_ld + r : r * pre_ld + k]) : v;
  }
  // This thread's share of: whether a block is flagged, of all or of those that
  // rows r0 .. r0 + n - 1 of this side lie in.
  __device__ __forceinline__ bool flagged() const {
    bool f = false;
    for (int i = threadIdx.x; i < flags_x * flags_y; i += blockDim.x) f |= flags[i] != 0;
    return f;
  }
  __device__ __forceinline__ bool flagged(int64_t r0, int n) const {
    const int64_t per = mn ? 1024 : rows_per;
    const int across = mn ? flags_y : flags_x, blocks = mn ? flags_x : flags_y;
    const int b0 = (int)(r0 / per), b1 = min((int)((r0 + n - 1) / per), blocks - 1);
    bool f = false;
    for (int b = b0; b <= b1; ++b)
      for (int i = threadIdx.x; i < across; i += blockDim.x)
        f |= flags[mn ? i * flags_x + b : b * flags_x + i] != 0;
    return f;
  }
};
struct NonFinite {
  Given a, b;
  int64_t M, N, K;
  Epilogue e;
};

// The results that infinities and NaN of the operands enter.  Such a result is an
// infinity or NaN, whatever the finite terms are, so only the terms with an operand
// that is not finite are summed; a chunk of K without any costs its loads.  Then the
// epilogue as in the product kernel, whose result, of the finite terms, stands in
// `out`: where that was the residual's memory it is taken for the residual, from
// which it differs by a finite value.  A tile of 32 x 32 results a CTA at a time,
// four a thread; blockIdx.y: the product.  Where nothing is flagged it ends at once
// (1 to 4 us of the call); 4095 x 2048 -> 4384 takes 0.64 ms instead of 0.28 with one
// infinity, 0.94 with nothing but NaN, 12 with an infinity late in every row.
constexpr int kFixTile = 32;
__global__ void __launch_bounds__(256)
    nonfinite_kernel(const __grid_constant__ NonFinite p0, const __grid_constant__ NonFinite p1) {
  const NonFinite& p = blockIdx.y == 0 ? p0 : p1;
  const bool some = p.a.flagged() | p.b.flagged();
  if (!__syncthreads_or(some)) return;
  __shared__ float sa[kFixTile][kFixTile + 1], sb[kFixTile][kFixTile + 1];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t tiles_n = (p.N + kFixTile - 1) / kFixTile;
  const int64_t tiles = (p.M + kFixTile - 1) / kFixTile * tiles_n;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t m0 = t / tiles_n * kFixTile, n0 = t % tiles_n * kFixTile;
    const int64_t n = n0 + tx;
    const bool here = p.a.flagged(m0, kFixTile) | p.b.flagged(n0, kFixTile);
    if (!__syncthreads_or(here)) continue;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    bool open = true;   // (a NaN stays one: a tile of them is done)
    for (int64_t k0 = 0; __syncthreads_or(open) && k0 < p.K; k0 += kFixTile) {
      bool found = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {   // consecutive threads, consecutive addresses
        const int y = ty + 8 * i;
        const int ra = p.a.mn ? tx : y, ka = p.a.mn ? y : tx;
        const int rb = p.b.mn ? tx : y, kb = p.b.mn ? y : tx;
        const float a = m0 + ra < p.M && k0 + ka < p.K ? p.a.at(m0 + ra, k0 + ka) : 0.f;
        const float b = n0 + rb < p.N && k0 + kb < p.K ? p.b.at(n0 + rb, k0 + kb) : 0.f;
        found |= !isfinite(a) || !isfinite(b);
        sa[ra][ka] = a;
        sb[rb][kb] = b;
      }
      if (!__syncthreads_or(found)) continue;
      for (int k = 0; k < kFixTile && k0 + k < p.K; ++k) {
        const float b = sb[tx][k];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = sa[ty + 8 * i][k];
          if (!isfinite(a) || !isfinite(b)) acc[i] += a * b;
        }
      }
      open = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) open |= m0 + ty + 8 * i < p.M && n < p.N && !isnan(acc[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = m0 + ty + 8 * i;
      if (m >= p.M || n >= p.N || isfinite(acc[i])) continue;
      float v = acc[i];
      if (p.e.bias) v += get1(p.e.bias, p.e.bias_t, n);
      if (p.e.pre) put1(p.e.pre, p.e.pre_t, m * p.N + n, v);
      v = act_f(p.e.act, v);
      if (p.e.res) v += get1(p.e.res, p.e.res_t, m * p.e.res_ld + n);
      put1(p.e.out, p.e.out_t, m * p.e.out_ld + n, v);
    }
  }
}

// out[c] = sum over r of part[r][c], rounded once to out's type.
__global__ void __launch_bounds__(256)
    sum_rows_kernel(const float* __restrict__ part, int rows, int C, void* out, int out_t) {
  __shared__ float acc[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < C) {
#pragma unroll 8
    for (int r = w; r < rows; r += 8) s += part[(int64_t)r * C + c];
  }
  acc[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < C) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += acc[i][lane];
    put1(out, out_t, c, s);
  }
}

// ------------------------------------------------------------------- few rows

constexpr int kSkinnyThreads = 256, kSkinnyWarps = 8;   // (16 warps for few rows of W)

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 rows of W a CTA against NT x 8 tokens.  The warps take steps of 32 of K
// in turn.  Each lane loads 16 consecutive bytes of a row: the MMA's K index
// is permuted within the step, alike for W and x, which leaves the sum as it
// is.  K a multiple of 8, rows 16-byte aligned.
template <int NT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32)
    skinny_bf16_kernel(const __nv_bfloat16* __restrict__ x, int64_t sx,
                       const __nv_bfloat16* __restrict__ w, int M, int64_t N, int K,
                       const __grid_constant__ Epilogue e) {
  __shared__ float acc[WARPS][16][NT * 8 + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const bool lo = n0 + g < N, hi = n0 + g + 8 < N;
  const __nv_bfloat16* w0 = w + (n0 + g) * K;
  const __nv_bfloat16* w1 = w0 + (int64_t)8 * K;
  float d[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) d[i][j] = 0.f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 4
  for (int k = (warp * 4 + t) * 8; k < K + t * 8; k += WARPS * 32) {   // uniform trip count
    const bool in = k < K;
    const uint4 a = in && lo ? *reinterpret_cast<const uint4*>(w0 + k) : zero;
    const uint4 b = in && hi ? *reinterpret_cast<const uint4*>(w1 + k) : zero;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int m = i * 8 + g;
      const uint4 v = in && m < M ? *reinterpret_cast<const uint4*>(x + m * sx + k) : zero;
      mma16816(d[i], a.x, b.x, a.y, b.y, v.x, v.y);
      mma16816(d[i], a.z, b.z, a.w, b.w, v.z, v.w);
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    acc[warp][g][i * 8 + 2 * t] = d[i][0];
    acc[warp][g][i * 8 + 2 * t + 1] = d[i][1];
    acc[warp][g + 8][i * 8 + 2 * t] = d[i][2];
    acc[warp][g + 8][i * 8 + 2 * t + 1] = d[i][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < NT * 8 * 4; i += WARPS * 32) {
    const int m = i >> 2, c = (i & 3) * 4;
    if (m >= M) continue;
    float v[4] = {0.f, 0.f, 0.f, 0.f}, res[4];
    residual4(e, m, n0 + c, N, res);
#pragma unroll
    for (int q = 0; q < WARPS; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += acc[q][c + j][m];
    finish4(e, m, n0 + c, N, v, res);
  }
}

// fp32: a CTA takes four rows of W against 8 tokens, its warps steps of
// 128 of K in turn (so that x is read once a CTA).  The 32 sums are folded over
// the lanes: each halving keeps half of them in either half of the lanes, and
// lane m * 4 + j ends up with token m, row j.  K a multiple of 4, rows 16-byte
// aligned.
constexpr int kF32Rows = 4;
__global__ void __launch_bounds__(kSkinnyThreads)
    skinny_f32_kernel(const float* __restrict__ x, int64_t sx, const float* __restrict__ w, int M,
                      int64_t N, int K, const __grid_constant__ Epilogue e) {
  __shared__ float part[kSkinnyWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t n0 = (int64_t)blockIdx.x * kF32Rows, m0 = (int64_t)blockIdx.y * 8;
  x += m0 * sx;
  M -= (int)m0;
  float acc[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) acc[i] = 0.f;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = (warp * 32 + lane) * 4; k < K; k += kSkinnyWarps * 128) {
    float4 wv[kF32Rows], xv[8];
#pragma unroll
    for (int j = 0; j < kF32Rows; ++j)
      wv[j] = n0 + j < N ? *reinterpret_cast<const float4*>(w + (n0 + j) * K + k) : zero;
#pragma unroll
    for (int m = 0; m < 8; ++m)
      xv[m] = m < M ? *reinterpret_cast<const float4*>(x + m * sx + k) : zero;
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int j = 0; j < kF32Rows; ++j) {
        float& a = acc[m * 4 + j];
        a = fmaf(xv[m].x, wv[j].x, a);
        a = fmaf(xv[m].y, wv[j].y, a);
        a = fmaf(xv[m].z, wv[j].z, a);
        a = fmaf(xv[m].w, wv[j].w, a);
      }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < off; ++i) {
      const float keep = up ? acc[i + off] : acc[i], give = up ? acc[i] : acc[i + off];
      acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
    }
  }
  part[warp][lane] = acc[0];
  __syncthreads();
  if (warp > 0) return;
  float v = 0.f;
#pragma unroll
  for (int q = 0; q < kSkinnyWarps; ++q) v += part[q][lane];
  const int64_t m = m0 + (lane >> 2), n = n0 + (lane & 3);
  if ((lane >> 2) >= M || n >= N) return;
  if (e.bias) v += get1(e.bias, e.bias_t, n);
  if (e.pre) put1(e.pre, e.pre_t, m * N + n, v);
  v = act_f(e.act, v);
  if (e.res) v += get1(e.res, e.res_t, m * e.res_ld + n);
  put1(e.out, e.out_t, m * e.out_ld + n, v);
}

// ------------------------------------------------------------------- host side

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

int bad(int code, const char* msg) { return set_error(code, msg); }
int cuda_bad(cudaError_t e, const char* what) {
  char m[256];
  snprintf(m, sizeof(m), "%s: %s", what, cudaGetErrorString(e));
  return set_error(SSD_ERR_CUDA, m);
}
bool al(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// An operand in memory: `rows` rows of `cols` bf16, ld apart, `planes` of them
// rows * ld apart.
struct Operand {
  const void* p;
  int64_t rows, cols, ld;
  int planes;
};

// box: kBK x tile rows of a K-major operand, 64 x kBK of an MN-major one.
bool make_map(CUtensorMap* m, const Operand& o, bool mn, int tile_rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  // Loads from a map of less than 128 KB are slower (M = 17, K = 2560, N = 10576:
  // 31 us instead of 24), so a small operand's map is given a second plane past
  // that size, which no load's coordinates reach.
  const bool small = o.planes == 1 && o.rows * o.ld * 2 < 131072;
  const cuuint64_t dims[3] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows,
                              (cuuint64_t)(small ? 2 : o.planes)};
  const cuuint64_t strides[2] = {
      (cuuint64_t)o.ld * 2,
      (cuuint64_t)(small ? 131072 : o.planes > 1 ? o.rows * o.ld * 2 : o.ld * 2)};
  const cuuint32_t box[3] = {64, (cuuint32_t)(mn ? kBK : tile_rows), 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(o.p), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a product of M x N with `steps` K steps is cut: CTAs a tile, tile width,
// the tiles computed whole, and the splits of K of the others.
struct Plan {
  int cg, bn, full, tail, splits, steps_per;
  size_t partial_bytes() const {
    return splits > 1 ? (size_t)tail * splits * cg * kBM * bn * sizeof(float) : 0;
  }
};
// A model of its time in microseconds, over all tile widths (multiples of 32).
// Tiles fill the SMs in rounds; the last, incomplete round's tiles may be split
// along K over the SMs that it would leave idle (dx of 4096 x 10576 -> 2560: 160
// tiles on 76 pairs), in one round of splits or several (8192 rows: 16 tiles
// left in four splits, 247 us instead of 271).  A K step takes the tensor cores
// 2 BN cycles, the shared memory the time to write and read the step's tiles at
// 128 bytes a cycle (measured: 528 cycles for 256 x 256 on a pair, 524 for
// 128 x 128 on one CTA), and the MMA warp 350 to 400 cycles to issue.
Plan plan_for(int64_t M, int64_t N, int64_t K, int pairs, bool bmn) {
  const int sms = row::sm_count();
  const int steps = (int)((K + kBK - 1) / kBK) * pairs;
  constexpr double kGhz = 1.9, kL2Gbs = 20e3, kHbmGbs = 6e3, kJoinUs = 8.0, kJoinGbs = 5e3;
  const double hbm_us = ((double)(M + N) * K * 2 * (pairs > 1 ? 3 : 1)) / kHbmGbs * 1e-3;
  Plan best = {2, 256, 1, 0, 1, steps};
  double best_us = 1e30;
  for (int cg = 1; cg <= 2; ++cg) {
    for (int bn = 32; bn <= 256; bn += 32) {
      if (bmn && bn % (64 * cg) != 0) continue;   // whole blocks of an MN-major B
      const int64_t tiles = ((M + kBM * cg - 1) / (kBM * cg)) * ((N + bn - 1) / bn);
      const double step_bytes = kStageA + stage_b(cg, bn, bmn);   // a CTA's
      const double step = std::max({2.0 * bn, 2.0 * step_bytes / 128, 380.0}) * 1e-3 / kGhz;
      const int64_t at_once = sms / cg, rounds = tiles / at_once, tail = tiles % at_once;
      const double l2_us = tiles * steps * step_bytes * cg / kL2Gbs * 1e-3;
      for (int splits = 1; splits <= 16; ++splits) {
        const int per = (steps + splits - 1) / splits;
        if (splits > 1 && (tail == 0 || per < 8 || (steps + per - 1) / per != splits)) continue;
        const int64_t parts = (tail * splits + at_once - 1) / at_once;   // rounds of splits
        double us = (rounds * steps + parts * per) * step;
        us = std::max(std::max(us, l2_us), hbm_us) + 3.0 + 2.0 * bn / 256;   // fill, last epilogue
        // partial sums are written, read and joined by another launch
        if (splits > 1)
          us += kJoinUs + (double)tail * cg * kBM * bn * splits * 8 / kJoinGbs * 1e-3;
        if (us < best_us) {
          best_us = us;
          best = {cg, bn, (int)(splits > 1 ? tiles - tail : tiles), (int)(splits > 1 ? tail : 0),
                  splits, per};
        }
      }
    }
  }
  return best;
}

// Persistent CTAs (or pairs) of a kernel that fit the device at once, cached
// per device; the first call also opts in to its shared memory.
template <int CG, bool AMN, bool BMN, bool EXACT, bool PLAIN>
cudaError_t resident(int* n) {
  static std::atomic<int> cached[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < 64;
  *n = known ? cached[dev].load(std::memory_order_acquire) : 0;
  if (*n > 0) return cudaSuccess;
  const size_t smem = sizeof(Smem) + 1024;
  auto* kernel = gemm_kernel<CG, AMN, BMN, EXACT, PLAIN>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  *n = row::sm_count() / CG;
  if (CG > 1) {   // some SMs may have no partner
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(row::sm_count() / CG * CG);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = CG;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int most = 0;
    e = cudaOccupancyMaxActiveClusters(&most, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (most > 0) *n = std::min(*n, most);
  }
  if (known) cached[dev].store(*n, std::memory_order_release);
  return cudaSuccess;
}

template <int CG, bool AMN, bool BMN, bool EXACT, bool PLAIN>
cudaError_t launch_gemm(const CUtensorMap& ma, const CUtensorMap& mb, const Gemm& g,
                        cudaStream_t st) {
  int at_once = 0;
  const cudaError_t e = resident<CG, AMN, BMN, EXACT, PLAIN>(&at_once);
  if (e != cudaSuccess) return e;
  const int64_t items = g.full + ((int64_t)g.tiles_m * g.tiles_n - g.full) * g.splits;
  const int grid = CG * (int)std::min<int64_t>(items, at_once);
  gemm_kernel<CG, AMN, BMN, EXACT, PLAIN>
      <<<grid, kThreads, sizeof(Smem) + 1024, st>>>(ma, mb, g);
  return cudaGetLastError();
}

// D[M,N] = sum over K and planes, finished by e; part: the plan's partial_bytes.
int gemm(const Operand& a, bool amn, const Operand& b, bool bmn, int64_t M, int64_t N, int64_t K,
         const Epilogue& e, float* part, cudaStream_t st) {
  const int pairs = a.planes == 3 ? 6 : 1;
  const Plan pl = plan_for(M, N, K, pairs, bmn);
  CUtensorMap ma, mb;
  if (!make_map(&ma, a, amn, kBM) || !make_map(&mb, b, bmn, rows_b(pl.cg, pl.bn, bmn)))
    return bad(SSD_ERR_CUDA, "linear: a tensor map could not be made");
  Gemm g = {};
  g.M = M;
  g.N = N;
  g.kblocks = (int)((K + kBK - 1) / kBK);
  g.pairs = pairs;
  g.tiles_m = (int)((M + kBM * pl.cg - 1) / (kBM * pl.cg));
  g.tiles_n = (int)((N + pl.bn - 1) / pl.bn);
  g.full = pl.full;
  g.splits = pl.splits;
  g.steps_per_split = pl.steps_per;
  g.bn = pl.bn;
  g.stages = std::min(kMaxStages, kOperandBytes / (kStageA + stage_b(pl.cg, pl.bn, bmn)));
  g.group_m = 8 / pl.cg;
  // runs of the longest item's K steps
  const int longest = pl.full > 0 ? g.kblocks * pairs : pl.steps_per;
  const bool exact = e.out_t == kF32 || longest > kBf16Steps;
  g.run = pairs == 1 ? kExactSteps : kPlanesSteps;
  g.lead = (pairs - 1) * g.kblocks;
  if (e.out_t != kF32) {   // as even as they can be
    const int runs = (longest + kBf16Steps - 1) / kBf16Steps;
    g.run = (longest + runs - 1) / runs;
  }
  g.partial = part;
  g.e = e;
  const bool plain = !e.bias && !e.pre && !e.res && e.act == kActNone;
  cudaError_t err;
  // (the backward's products are plain)
#define SSD_GEMM_AS(CG, EXACT)                                                               \
  err = amn   ? launch_gemm<CG, true, true, EXACT, true>(ma, mb, g, st)                      \
        : bmn ? launch_gemm<CG, false, true, EXACT, true>(ma, mb, g, st)                     \
        : plain ? launch_gemm<CG, false, false, EXACT, true>(ma, mb, g, st)                  \
                : launch_gemm<CG, false, false, EXACT, false>(ma, mb, g, st)
  if (pl.cg == 2 && exact) SSD_GEMM_AS(2, true);
  else if (pl.cg == 2) SSD_GEMM_AS(2, false);
  else if (exact) SSD_GEMM_AS(1, true);
  else SSD_GEMM_AS(1, false);
#undef SSD_GEMM_AS
  if (err != cudaSuccess) return cuda_bad(err, "linear launch");
  if (pl.splits > 1) {
    const int rows = kBM * pl.cg;
    join_kernel<<<dim3((unsigned)((rows * pl.bn / 4 + 255) / 256), (unsigned)pl.tail), 256, 0, st>>>(
        g, rows);
    err = cudaGetLastError();
    if (err != cudaSuccess) return cuda_bad(err, "linear join launch");
  }
  return SSD_OK;
}

int type_of(ssd_dtype_t t) { return t == SSD_DTYPE_BF16 ? kBf16 : kF32; }
size_t esize(ssd_dtype_t t) { return t == SSD_DTYPE_BF16 ? 2 : 4; }

// Rows of a plane / column-sum pass a CTA: about eight CTAs of 128 threads an
// SM; bounded by the grid's y limit.
int64_t prep_rows_per(int64_t R, int C) {
  const int64_t cols = (C + 1023) / 1024;
  const int64_t want = std::max<int64_t>(1, (int64_t)row::sm_count() * 8 / cols);
  return std::max<int64_t>(std::max<int64_t>(4, (R + want - 1) / want), (R + 65534) / 65535);
}
int64_t prep_parts(int64_t R, int C) {
  const int64_t per = prep_rows_per(R, C);
  return (R + per - 1) / per;
}
int64_t padded(int64_t c) { return (c + 7) & ~(int64_t)7; }
size_t planes_bytes(int64_t R, int64_t C, int planes) {
  return up256((size_t)planes * R * padded(C) * 2);
}

// src as operand planes at `out`; column sums to colsum if not null.
cudaError_t prep(const void* src, int src_t, int64_t ld, int64_t R, int C, const void* pre, int pre_t,
                 int act, int planes, void* out, float* colsum, int* flags, cudaStream_t st) {
  Prep p = {};
  p.flags = planes == 3 ? flags : nullptr;
  p.src = src;
  p.pre = pre;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.colsum = colsum;
  p.R = R;
  p.src_ld = ld;
  p.ld = padded(C);
  p.rows_per = prep_rows_per(R, C);
  p.C = C;
  p.src_t = (uint8_t)src_t;
  p.pre_t = (uint8_t)pre_t;
  p.act = (uint8_t)act;
  p.planes = (uint8_t)planes;
  const unsigned parts = (unsigned)prep_parts(R, C);
  const dim3 grid((unsigned)((C + 1023) / 1024), parts);
  if (C % 8 == 0 && ld % 8 == 0 && al(src, 16) && al(pre, 16))
    (planes == 3 ? prep_kernel<false, true> : prep_kernel<false, false>)<<<grid, 128, 0, st>>>(p);
  else
    (planes == 3 ? prep_kernel<true, true> : prep_kernel<true, false>)<<<grid, 128, 0, st>>>(p);
  return cudaGetLastError();
}

// The flags of an fp32 operand's prep_kernel blocks.
size_t flags_bytes(int64_t R, int64_t C) {
  return up256(sizeof(int) * (size_t)prep_parts(R, (int)C) * ((C + 1023) / 1024));
}
// An operand of R rows of C for nonfinite_kernel.
Given given(const void* src, int64_t R, int64_t C, int64_t ld, const int* flags, bool mn) {
  Given g = {};
  g.src = static_cast<const float*>(src);
  g.flags = flags;
  g.ld = ld;
  g.rows_per = prep_rows_per(R, (int)C);
  g.flags_x = (int)((C + 1023) / 1024);
  g.flags_y = (int)prep_parts(R, (int)C);
  g.mn = mn;
  return g;
}
// Puts what infinities and NaN of fp32 operands contribute into the results of one
// product or two.
cudaError_t fix_nonfinite(const NonFinite* p, int products, cudaStream_t st) {
  int64_t tiles = 0;
  for (int i = 0; i < products; ++i)
    tiles = std::max(tiles, ((p[i].M + kFixTile - 1) / kFixTile) *
                                ((p[i].N + kFixTile - 1) / kFixTile));
  const dim3 grid((unsigned)std::min<int64_t>(tiles, row::sm_count()), (unsigned)products);
  nonfinite_kernel<<<grid, 256, 0, st>>>(p[0], p[products - 1]);
  return cudaGetLastError();
}

int check_sizes(int64_t rows, int in_f, int out_f, ssd_dtype_t dt) {
  if (dt != SSD_DTYPE_F32 && dt != SSD_DTYPE_BF16) return bad(SSD_ERR_ARG, "unknown dtype");
  if (rows < 1 || in_f < 1 || out_f < 1)
    return bad(SSD_ERR_ARG, "rows, in_features and out_features must be >= 1");
  if (rows > (1LL << 30) || in_f > (1 << 24) || out_f > (1 << 24))
    return bad(SSD_ERR_UNSUPPORTED, "rows above 2^30 or features above 2^24");
  // tiles (of 128 x 64) are counted in 31 bits
  for (const int64_t t : {((rows + 127) / 128) * ((int64_t)(std::max(in_f, out_f) + 63) / 64),
                          (((int64_t)out_f + 127) / 128) * (((int64_t)in_f + 63) / 64)})
    if (t * 16 > 0x7fffffff) return bad(SSD_ERR_UNSUPPORTED, "the product is too large");
  return SSD_OK;
}

// Whether a bf16 matrix can be read by TMA where it lies.
bool in_place(const void* p, int64_t ld, ssd_dtype_t dt) {
  return dt == SSD_DTYPE_BF16 && al(p, 16) && ld % 8 == 0 && ld < (1LL << 38);
}

// Whether the weight is streamed through registers.  bf16: every CTA reads all of
// x, so beyond 8 rows x has to be small (64 KB): 16 rows x 1024 -> 1024 take 9 us
// here and 15 in the product kernel, 16 x 2560 -> 10576 take 26 and 23.  fp32, whose
// product kernel wants both operands split first: a pass over the weight for each
// 8 rows, up to 24 rows (16 x 2560 -> 10576: 75 us instead of 112, 32 rows: 132 and
// 112), or up to 128 where the passes are short, by the cost of their CTAs of four
// outputs (64 x 1024 -> 1024: 22 and 24, 128 x 512 -> 352: 16 and 26, 96 x 1024 ->
// 1024: 28 and 24; 1000 x 64 -> 64: 20 and 16).  (All with 5 to 10 us of measuring
// around them.)
constexpr int kSkinnyBf16 = 32, kSkinnyF32 = 24, kSkinnyMax = 128;
bool few_rows(int64_t rows, int K, int64_t N, ssd_dtype_t dt) {
  if (dt == SSD_DTYPE_F32)
    return rows <= kSkinnyF32 || (rows <= kSkinnyMax &&
                                  ((rows + 7) / 8) * ((N + 3) / 4) * (K + 512) <= 3000000);
  return rows <= 8 || (rows <= kSkinnyBf16 && rows * K <= 32768);
}

bool skinny(const void* x, int64_t sx, const void* w, int64_t rows, int K, int64_t N,
            ssd_dtype_t dt) {
  const int unit = dt == SSD_DTYPE_BF16 ? 8 : 4;   // elements of a 16-byte load
  return few_rows(rows, K, N, dt) && K % unit == 0 && al(x, 16) && al(w, 16) &&
         (rows == 1 || sx % unit == 0);
}

// every row of a tensor starts on a multiple of four elements
bool wide4(const void* p, int64_t ld, size_t e) { return al(p, 4 * e) && ld % 4 == 0; }

size_t fwd_bytes(int64_t rows, int K, int N, ssd_dtype_t dt, bool pack_x, bool pack_w) {
  const int planes = dt == SSD_DTYPE_F32 ? 3 : 1;
  size_t b = up256(plan_for(rows, N, K, planes == 3 ? 6 : 1, false).partial_bytes());
  if (pack_x) b += planes_bytes(rows, K, planes);
  if (pack_w) b += planes_bytes(N, K, planes);
  if (planes == 3) b += flags_bytes(rows, K) + flags_bytes(N, K);
  return b;
}
size_t bwd_bytes(int64_t rows, int K, int N, ssd_dtype_t dt, bool pack_x, bool pack_w, bool pack_d) {
  const int planes = dt == SSD_DTYPE_F32 ? 3 : 1, pairs = planes == 3 ? 6 : 1;
  size_t b = up256(std::max(plan_for(rows, K, N, pairs, true).partial_bytes(),
                            plan_for(N, K, rows, pairs, true).partial_bytes()));
  b += up256((size_t)prep_parts(rows, N) * N * sizeof(float));
  if (pack_x) b += planes_bytes(rows, K, planes);
  if (pack_w) b += planes_bytes(N, K, planes);
  if (pack_d) b += planes_bytes(rows, N, planes);
  if (planes == 3) b += flags_bytes(rows, N) + flags_bytes(N, K) + flags_bytes(rows, K);
  return b;
}

}  // namespace linear

int linear_status(int reset, cudaStream_t st, int* bits) {
  int h = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&h, linear::g_status_linear, sizeof(int), 0,
                                            cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && reset && h != 0) {
    static const int zero = 0;
    e = cudaMemcpyToSymbolAsync(linear::g_status_linear, &zero, sizeof(int), 0,
                                cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  *bits = h;
  return (int)e;
}

}  // namespace ssd

using namespace ssd;
using namespace ssd::linear;

extern "C" {

size_t ssd_linear_fwd_workspace_bytes(int64_t rows, int in_features, int out_features,
                                      ssd_dtype_t dtype, int aligned) {
  if (check_sizes(rows, in_features, out_features, dtype) != SSD_OK) return 0;
  const bool odd = !aligned || in_features % 8 != 0;
  if (!odd && few_rows(rows, in_features, out_features, dtype)) return 0;
  // (a strided x may be aligned while a weight of odd rows is not: the sum is enough for both)
  const bool pack = dtype == SSD_DTYPE_F32 || odd;
  return fwd_bytes(rows, in_features, out_features, dtype, pack, pack);
}

int ssd_linear_fwd(const void* x, int64_t x_row_stride, const void* weight, const void* bias,
                   const void* residual, int64_t residual_row_stride, int64_t rows, int in_features,
                   int out_features, ssd_activation_t activation, ssd_dtype_t dtype,
                   ssd_dtype_t residual_dtype, void* out, void* pre, void* workspace,
                   size_t workspace_bytes, void* stream) {
  const int c = check_sizes(rows, in_features, out_features, dtype);
  if (c != SSD_OK) return c;
  if (activation < SSD_ACT_NONE || activation > SSD_ACT_GELU)
    return bad(SSD_ERR_ARG, "unknown activation");
  if (residual && residual_dtype != dtype && residual_dtype != SSD_DTYPE_F32)
    return bad(SSD_ERR_ARG, "the residual is fp32 or of the x dtype");
  if (!x || !weight || !out) return bad(SSD_ERR_NULL, "x, weight and out are required");
  const size_t e = esize(dtype), re = residual ? esize(residual_dtype) : e;
  if (!al(x, e) || !al(weight, e) || !al(bias, e) || !al(residual, re) || !al(out, re) ||
      !al(pre, dtype == SSD_DTYPE_BF16 ? 2 : 4))
    return bad(SSD_ERR_ALIGN, "a pointer is not aligned to its element");
  if (rows > 1 && (x_row_stride < in_features || (residual && residual_row_stride < out_features) ||
                   x_row_stride > (1LL << 40) || residual_row_stride > (1LL << 40)))
    return bad(SSD_ERR_ARG, "row strides must be at least the features, and below 2^40");
  const int64_t K = in_features, N = out_features;
  const int64_t sx = rows > 1 ? x_row_stride : padded(K);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Epilogue ep = {};
  ep.bias = bias;
  ep.bias_t = (uint8_t)type_of(dtype);
  ep.res = residual;
  ep.res_t = (uint8_t)type_of(residual_dtype);
  ep.res_ld = rows > 1 ? residual_row_stride : padded(N);
  ep.out = out;
  ep.out_t = (uint8_t)type_of(residual ? residual_dtype : dtype);
  ep.out_ld = N;
  ep.pre = pre;
  ep.pre_t = dtype == SSD_DTYPE_BF16 ? kF16 : kF32;
  ep.act = (uint8_t)act_of(activation, dtype);
  ep.wide = N % 4 == 0 && al(bias, 4 * e) && al(out, 4 * re) &&
            al(pre, dtype == SSD_DTYPE_BF16 ? 8 : 16) &&
            (!residual || wide4(residual, ep.res_ld, re));
  ep.wide8 = N % 8 == 0 && al(bias, 16) && al(out, 16) && al(pre, 16) &&
             (!residual || (al(residual, 16) && ep.res_ld % 8 == 0));
  if (skinny(x, sx, weight, rows, in_features, N, dtype)) {
    if (dtype == SSD_DTYPE_BF16) {
      const auto* xb = static_cast<const __nv_bfloat16*>(x);
      const auto* wb = static_cast<const __nv_bfloat16*>(weight);
      const unsigned grid = (unsigned)((N + 15) / 16);
      // one or two CTAs an SM: twice the warps, for the loads in flight (8 x 5120 ->
      // 2560: 17.5 us instead of 22.7; with more CTAs 8 warps are enough)
      const bool few = N < 16 * 2 * (int64_t)row::sm_count();
#define SSD_SKINNY(NT)                                                                          \
  if (few)                                                                                      \
    skinny_bf16_kernel<NT, 16><<<grid, 512, 0, st>>>(xb, sx, wb, (int)rows, N, in_features, ep); \
  else                                                                                          \
    skinny_bf16_kernel<NT, 8><<<grid, 256, 0, st>>>(xb, sx, wb, (int)rows, N, in_features, ep)
      if (rows <= 8) {
        SSD_SKINNY(1);
      } else if (rows <= 16) {
        SSD_SKINNY(2);
      } else {
        SSD_SKINNY(4);
      }
#undef SSD_SKINNY
    } else {
      const dim3 grid((unsigned)((N + kF32Rows - 1) / kF32Rows), (unsigned)((rows + 7) / 8));
      skinny_f32_kernel<<<grid, kSkinnyThreads, 0, st>>>(static_cast<const float*>(x), sx,
                                                         static_cast<const float*>(weight),
                                                         (int)rows, N, in_features, ep);
    }
    const cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? SSD_OK : cuda_bad(err, "linear launch");
  }
  const bool pack_x = !in_place(x, sx, dtype), pack_w = !in_place(weight, K, dtype);
  if (!al(workspace, 256)) return bad(SSD_ERR_ALIGN, "workspace: 256-byte aligned");
  const size_t need = fwd_bytes(rows, in_features, out_features, dtype, pack_x, pack_w);
  if (need > 0 && !workspace) return bad(SSD_ERR_NULL, "workspace is required");
  if (workspace_bytes < need) return bad(SSD_ERR_WORKSPACE, "workspace too small");
  const int planes = dtype == SSD_DTYPE_F32 ? 3 : 1;
  char* ws = static_cast<char*>(workspace);
  Operand a = {x, rows, K, sx, 1}, b = {weight, N, K, K, 1};
  int *fx = nullptr, *fw = nullptr;
  if (planes == 3) {
    fx = reinterpret_cast<int*>(ws);
    ws += flags_bytes(rows, K);
    fw = reinterpret_cast<int*>(ws);
    ws += flags_bytes(N, K);
  }
  if (pack_x) {
    const cudaError_t err = prep(x, type_of(dtype), sx, rows, in_features, nullptr, 0, 0, planes, ws,
                                 nullptr, fx, st);
    if (err != cudaSuccess) return cuda_bad(err, "linear operand launch");
    a = {ws, rows, K, padded(K), planes};
    ws += planes_bytes(rows, K, planes);
  }
  if (pack_w) {
    const cudaError_t err = prep(weight, type_of(dtype), K, N, in_features, nullptr, 0, 0, planes,
                                 ws, nullptr, fw, st);
    if (err != cudaSuccess) return cuda_bad(err, "linear operand launch");
    b = {ws, N, K, padded(K), planes};
    ws += planes_bytes(N, K, planes);
  }
  const int r = gemm(a, false, b, false, rows, N, K, ep, reinterpret_cast<float*>(ws), st);
  if (r != SSD_OK || planes != 3) return r;
  const NonFinite fix = {given(x, rows, K, sx, fx, false), given(weight, N, K, K, fw, false),
                         rows, N, K, ep};
  const cudaError_t err = fix_nonfinite(&fix, 1, st);
  return err == cudaSuccess ? SSD_OK : cuda_bad(err, "linear launch");
}

size_t ssd_linear_bwd_workspace_bytes(int64_t rows, int in_features, int out_features,
                                      ssd_dtype_t dtype, int aligned, int dout_as_is) {
  if (check_sizes(rows, in_features, out_features, dtype) != SSD_OK) return 0;
  const bool pack = dtype == SSD_DTYPE_F32 || !aligned;
  return std::max<size_t>(
      256, bwd_bytes(rows, in_features, out_features, dtype, pack || in_features % 8 != 0,
                     pack || in_features % 8 != 0, pack || !dout_as_is || out_features % 8 != 0));
}

int ssd_linear_bwd(const void* dout, ssd_dtype_t dout_dtype, const void* x, int64_t x_row_stride,
                   const void* weight, const void* pre, int64_t rows, int in_features,
                   int out_features, ssd_activation_t activation, ssd_dtype_t dtype, void* dx,
                   void* dweight, void* dbias, void* workspace, size_t workspace_bytes,
                   void* stream) {
  const int c = check_sizes(rows, in_features, out_features, dtype);
  if (c != SSD_OK) return c;
  if (activation < SSD_ACT_NONE || activation > SSD_ACT_GELU)
    return bad(SSD_ERR_ARG, "unknown activation");
  if (dout_dtype != dtype && dout_dtype != SSD_DTYPE_F32)
    return bad(SSD_ERR_ARG, "dout is fp32 or of the x dtype");
  const bool act = activation != SSD_ACT_NONE;
  if (!dout || (dweight && !x) || (dx && !weight) || (act && !pre) || !workspace)
    return bad(SSD_ERR_NULL,
               "dout and workspace, x for dweight, weight for dx and pre with an activation are "
               "required");
  const size_t e = esize(dtype);
  if (!al(dout, esize(dout_dtype)) || !al(x, e) || !al(weight, e) || !al(dx, e) || !al(dweight, e) ||
      !al(dbias, e) || !al(pre, dtype == SSD_DTYPE_BF16 ? 2 : 4) || !al(workspace, 256))
    return bad(SSD_ERR_ALIGN, "a pointer is not aligned to its element (workspace: 256 bytes)");
  if (rows > 1 && x && (x_row_stride < in_features || x_row_stride > (1LL << 40)))
    return bad(SSD_ERR_ARG, "row strides must be at least the features, and below 2^40");
  const int64_t K = in_features, N = out_features;
  const int64_t sx = rows > 1 ? x_row_stride : padded(K);
  const bool pack_x = dweight && !in_place(x, sx, dtype);
  const bool pack_w = dx && !in_place(weight, K, dtype);
  const bool products = dx || dweight;
  const bool pack_d = products && (act || dout_dtype != dtype || !in_place(dout, N, dtype));
  if (workspace_bytes < bwd_bytes(rows, in_features, out_features, dtype, pack_x, pack_w, pack_d))
    return bad(SSD_ERR_WORKSPACE, "workspace too small");
  const int planes = dtype == SSD_DTYPE_F32 ? 3 : 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  float* colsum = reinterpret_cast<float*>(ws);
  ws += up256((size_t)prep_parts(rows, out_features) * N * sizeof(float));
  Operand d = {dout, rows, N, N, 1}, w = {weight, N, K, K, 1}, xo = {x, rows, K, sx, 1};
  int *fd = nullptr, *fw = nullptr, *fx = nullptr;
  if (planes == 3) {
    fd = reinterpret_cast<int*>(ws);
    ws += flags_bytes(rows, N);
    fw = reinterpret_cast<int*>(ws);
    ws += flags_bytes(N, K);
    fx = reinterpret_cast<int*>(ws);
    ws += flags_bytes(rows, K);
  }
  if (pack_d || dbias) {
    const cudaError_t err =
        prep(dout, type_of(dout_dtype), N, rows, out_features, act ? pre : nullptr,
             dtype == SSD_DTYPE_BF16 ? kF16 : kF32, act_of(activation, dtype), pack_d ? planes : 0, ws,
             dbias ? colsum : nullptr, fd, st);
    if (err != cudaSuccess) return cuda_bad(err, "linear operand launch");
    if (pack_d) {
      d = {ws, rows, N, padded(N), planes};
      ws += planes_bytes(rows, N, planes);
    }
    if (dbias) {
      sum_rows_kernel<<<(unsigned)((N + 31) / 32), 256, 0, st>>>(
          colsum, (int)prep_parts(rows, out_features), out_features, dbias, type_of(dtype));
      const cudaError_t err2 = cudaGetLastError();
      if (err2 != cudaSuccess) return cuda_bad(err2, "linear dbias launch");
    }
  }
  if (pack_w) {
    const cudaError_t err = prep(weight, type_of(dtype), K, N, in_features, nullptr, 0, 0, planes,
                                 ws, nullptr, fw, st);
    if (err != cudaSuccess) return cuda_bad(err, "linear operand launch");
    w = {ws, N, K, padded(K), planes};
    ws += planes_bytes(N, K, planes);
  }
  if (pack_x) {
    const cudaError_t err = prep(x, type_of(dtype), sx, rows, in_features, nullptr, 0, 0, planes, ws,
                                 nullptr, fx, st);
    if (err != cudaSuccess) return cuda_bad(err, "linear operand launch");
    xo = {ws, rows, K, padded(K), planes};
    ws += planes_bytes(rows, K, planes);
  }
  Epilogue ep = {};
  ep.out_t = (uint8_t)type_of(dtype);
  ep.out_ld = K;
  float* part = reinterpret_cast<float*>(ws);
  NonFinite fix[2];
  int fixes = 0;
  Given gd = planes == 3 ? given(dout, rows, N, N, fd, false) : Given{};
  if (act) {
    gd.pre = static_cast<const float*>(pre);
    gd.pre_ld = N;
    gd.act = (uint8_t)activation;
  }
  if (dx) {
    ep.out = dx;
    ep.wide = K % 4 == 0 && al(dx, 4 * e);
    ep.wide8 = K % 8 == 0 && al(dx, 16);
    const int r = gemm(d, false, w, true, rows, K, N, ep, part, st);
    if (r != SSD_OK) return r;
    if (planes == 3) fix[fixes++] = {gd, given(weight, N, K, K, fw, true), rows, K, N, ep};
  }
  if (dweight) {
    ep.out = dweight;
    ep.wide = K % 4 == 0 && al(dweight, 4 * e);
    ep.wide8 = K % 8 == 0 && al(dweight, 16);
    const int r = gemm(d, true, xo, true, N, K, rows, ep, part, st);
    if (r != SSD_OK) return r;
    gd.mn = true;
    if (planes == 3) fix[fixes++] = {gd, given(x, rows, K, sx, fx, true), N, K, rows, ep};
  }
  if (fixes > 0) {
    const cudaError_t err = fix_nonfinite(fix, fixes, st);
    if (err != cudaSuccess) return cuda_bad(err, "linear launch");
  }
  return SSD_OK;
}

}  // extern "C"
