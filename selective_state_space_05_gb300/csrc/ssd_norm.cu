// RMSNorms of the block: with the residual stream before it, with the gate
// after its scan, forward and backward.
//
// Both are bound by HBM: a forward reads its inputs and writes its outputs
// once, and so does a backward, which keeps the row it normalises in
// registers, packed as it was loaded.  A team of threads (8 to 512) holds a row
// (add) or a channel group of a row (gated), eight elements to a slot and up to
// four slots a thread, so each statistic is one sum over the team, and a row
// that one warp holds needs no barrier.  With n = r * s,
// s = 1 / sqrt(mean r^2 + eps), g = w dy, the backward
//   dr = s (g - n mean(g n)) = s (g - r s^2 mean(g r))
// needs mean r^2 and mean g r, which are summed together: one exchange.
// The parameters' gradients sum over rows: each team walks rows a grid apart
// and keeps its columns' sums in registers, writes them once to the
// workspace, and launch_column_sum joins the teams in a fixed order.
//
// Measured on one GB300 (6.69 TB/s copy), 32768 rows: add_rmsnorm of 2560
// channels (bf16, fp32 residual) forward 149 us = 6.77 TB/s, backward with scale
// 274 us = 5.5 TB/s; gated_rmsnorm of 5120 channels (bf16) in 8 groups forward
// 193 us = 5.2 TB/s, backward 337 us = 5.0 TB/s, where it issues 70 % of the
// cycles: exponentials, reciprocals and the conversions of five operands.
#include <stdio.h>

#include <algorithm>
#include <atomic>

#include "../../include/ssd_block.h"
#include "ssd_common.cuh"
#include "ssd_row.cuh"

namespace ssd {
namespace row {

int sm_count() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    n = n > 0 ? n : 152;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace row

namespace norm {

using row::kVec;
using row::load_slot;
using row::Slot;
using row::store_slot;

constexpr int kMaxThreads = row::kRowThreads;

// ---------------------------------------------------------------- add_rmsnorm

template <typename T, typename R, bool VEC, int S>
__global__ void __launch_bounds__(kMaxThreads)
    add_fwd_kernel(const T* __restrict__ x, const R* residual, const float* __restrict__ scale,
                   const float* __restrict__ weight, float eps, uint32_t rows, int dim, int nt,
                   T* __restrict__ y, R* rout) {
  __shared__ row::TeamSums sums;
  const int team = threadIdx.x / nt, t = threadIdx.x % nt, teams = blockDim.x / nt;
  const int64_t r = (int64_t)blockIdx.x * teams + team;
  const bool live = r < rows;
  float v[S][kVec], ss[1] = {0.f};
  if (live) {
    Slot<T, VEC> xs[S];
    Slot<R, VEC> rs[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
      xs[s].load(x + r * dim, s, t, nt, dim);
      if (residual) rs[s].load(residual + r * dim, s, t, nt, dim);
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      xs[s].get(v[s]);
      if (scale) {
        float c[kVec];
        load_slot<VEC>(scale, s, t, nt, dim, c);
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[s][j] *= c[j];
      }
      if (residual) {
        float q[kVec];
        rs[s].get(q);
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[s][j] += q[j];
      }
      store_slot<VEC>(rout + r * dim, s, t, nt, dim, v[s]);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        v[s][j] = row::stored(v[s][j], (const R*)nullptr);
        ss[0] = fmaf(v[s][j], v[s][j], ss[0]);
      }
    }
  }
  row::team_sum(ss, sums, 0, team, nt);
  if (!live) return;
  const float rstd = rsqrtf(ss[0] / (float)dim + eps);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    float w[kVec];
    load_slot<VEC>(weight, s, t, nt, dim, w);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[s][j] = v[s][j] * rstd * w[j];
    store_slot<VEC>(y + r * dim, s, t, nt, dim, v[s]);
  }
}

// Partial sums of team q of the grid: part[q * 2 * dim + c] for dweight, and
// dim further for dscale.  All of a row's loads are in flight before its sums.
template <typename T, typename R, bool VEC, int S>
__global__ void __launch_bounds__(kMaxThreads)
    add_bwd_kernel(const T* __restrict__ dy, const R* dres_out, const R* __restrict__ rin,
                   const T* __restrict__ x, const float* __restrict__ scale,
                   const float* __restrict__ weight, float eps, uint32_t rows, int dim, int nt,
                   T* __restrict__ dx, R* dres, float* __restrict__ part) {
  __shared__ row::TeamSums sums;
  const int team = threadIdx.x / nt, t = threadIdx.x % nt, teams = blockDim.x / nt;
  float dw[S][kVec], ds[S][kVec];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int j = 0; j < kVec; ++j) dw[s][j] = ds[s][j] = 0.f;
  int buf = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * teams; r0 < rows; r0 += (int64_t)gridDim.x * teams) {
    const int64_t r = r0 + team;
    const bool live = r < rows;
    Slot<R, VEC> rs[S], dr[S];
    Slot<T, VEC> gs[S], xs[S];
    float c[2] = {0.f, 0.f};
    if (live) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        rs[s].load(rin + r * dim, s, t, nt, dim);
        gs[s].load(dy + r * dim, s, t, nt, dim);
        if (dres_out) dr[s].load(dres_out + r * dim, s, t, nt, dim);
        if (scale) xs[s].load(x + r * dim, s, t, nt, dim);
      }
#pragma unroll
      for (int s = 0; s < S; ++s) {
        float w[kVec], rv[kVec], g[kVec];
        load_slot<VEC>(weight, s, t, nt, dim, w);
        rs[s].get(rv);
        gs[s].get(g);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          c[0] = fmaf(rv[j], rv[j], c[0]);
          c[1] = fmaf(g[j] * w[j], rv[j], c[1]);
        }
      }
    }
    row::team_sum(c, sums, buf, team, nt);
    buf ^= 1;
    if (!live) continue;
    const float rstd = rsqrtf(c[0] / (float)dim + eps);
    const float k = rstd * rstd * (c[1] / (float)dim);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      float w[kVec], rv[kVec], g[kVec], d[kVec];
      load_slot<VEC>(weight, s, t, nt, dim, w);
      rs[s].get(rv);
      gs[s].get(g);
      if (dres_out) {
        dr[s].get(d);
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) d[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        dw[s][j] = fmaf(g[j], rv[j] * rstd, dw[s][j]);
        d[j] = fmaf(rstd, fmaf(-rv[j], k, g[j] * w[j]), d[j]);
      }
      if (dres) store_slot<VEC>(dres + r * dim, s, t, nt, dim, d);
      if (scale) {
        float xv[kVec], sc[kVec];
        xs[s].get(xv);
        load_slot<VEC>(scale, s, t, nt, dim, sc);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          ds[s][j] = fmaf(d[j], xv[j], ds[s][j]);
          d[j] *= sc[j];
        }
      }
      if (dx) store_slot<VEC>(dx + r * dim, s, t, nt, dim, d);
    }
  }
  float* p = part + ((int64_t)blockIdx.x * teams + team) * 2 * dim;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    store_slot<VEC>(p, s, t, nt, dim, dw[s]);
    if (scale) store_slot<VEC>(p + dim, s, t, nt, dim, ds[s]);
  }
}

// -------------------------------------------------------------- gated_rmsnorm

struct Rows {   // rows of [batch, seqlen, ...] views; seqlen 0: one stride (the token's) for all
  uint32_t rows, seqlen;
  TokStride y, z, dz;
};
__device__ __forceinline__ int64_t row_off(const TokStride& s, uint32_t r, uint32_t seqlen) {
  if (seqlen == 0) return r * s.t;
  const uint32_t b = r / seqlen;
  return (int64_t)b * s.b + (int64_t)(r - b * seqlen) * s.t;
}

// What the gate does: nothing (no z), before the norm, after it.
enum { kNoGate = 0, kGateFirst = 1, kNormFirst = 2 };

template <typename T, bool VEC, int S, int MODE>
__global__ void __launch_bounds__(kMaxThreads)
    gated_fwd_kernel(const T* y, const T* __restrict__ z, const float* __restrict__ weight,
                     float eps, Rows rw, int dim, int gs, int nt, T* out) {
  __shared__ row::TeamSums sums;
  const int team = threadIdx.x / nt, t = threadIdx.x % nt, teams = blockDim.x / nt;
  const int c0 = blockIdx.y * gs;
  const int64_t r = (int64_t)blockIdx.x * teams + team;
  const bool live = r < rw.rows;
  float v[S][kVec], gate[S][kVec], ss[1] = {0.f};
  if (live) {
    Slot<T, VEC> ys[S], zs[S];
    const T* yr = y + row_off(rw.y, (uint32_t)r, rw.seqlen) + c0;
    const T* zr = MODE != kNoGate ? z + row_off(rw.z, (uint32_t)r, rw.seqlen) + c0 : nullptr;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      ys[s].load(yr, s, t, nt, gs);
      if (MODE != kNoGate) zs[s].load(zr, s, t, nt, gs);
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      ys[s].get(v[s]);
      if (MODE != kNoGate) {
        zs[s].get(gate[s]);
#pragma unroll
        for (int j = 0; j < kVec; ++j) gate[s][j] *= row::sigmoid<T>(gate[s][j]);
        if (MODE == kGateFirst) {
#pragma unroll
          for (int j = 0; j < kVec; ++j) v[s][j] *= gate[s][j];
        }
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) ss[0] = fmaf(v[s][j], v[s][j], ss[0]);
    }
  }
  row::team_sum(ss, sums, 0, team, nt);
  if (!live) return;
  const float rstd = rsqrtf(ss[0] / (float)gs + eps);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    float w[kVec];
    load_slot<VEC>(weight + c0, s, t, nt, gs, w);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      v[s][j] = v[s][j] * rstd * w[j];
      if (MODE == kNormFirst) v[s][j] *= gate[s][j];
    }
    store_slot<VEC>(out + r * dim + c0, s, t, nt, gs, v[s]);
  }
}

// With e = silu(z) (1 without z), e' its derivative, s = 1 / rms:
//   gate first:  u = y e,  g = w dout,  du = s (g - u s^2 mean(g u)),
//                dy = du e,  dz = du y e',  dw = sum dout u s
//   norm first:  g = w dout e,  dy = s (g - y s^2 mean(g y)),
//                dz = dout w y s e',  dw = sum dout e y s
// Partial dweight of team q of the grid's x: part[q * dim + c].  The operands
// stay packed and the sigmoid is taken twice: holding its fp32 values as well
// would halve the rows in flight.
template <typename T, bool VEC, int S, int MODE>
__global__ void __launch_bounds__(kMaxThreads, S == 1 ? 2 : 1)   // (one slot: 64 registers)
    gated_bwd_kernel(const T* __restrict__ dout, const T* __restrict__ y, const T* __restrict__ z,
                     const float* __restrict__ weight, float eps, Rows rw, int dim, int gs,
                     int nt, T* __restrict__ dy, T* __restrict__ dz,
                     float* __restrict__ part) {
  __shared__ row::TeamSums sums;
  const int team = threadIdx.x / nt, t = threadIdx.x % nt, teams = blockDim.x / nt;
  const int c0 = blockIdx.y * gs;
  float dw[S][kVec];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int j = 0; j < kVec; ++j) dw[s][j] = 0.f;
  int buf = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * teams; r0 < rw.rows;
       r0 += (int64_t)gridDim.x * teams) {
    const int64_t r = r0 + team;
    const bool live = r < rw.rows;
    Slot<T, VEC> ys[S], zs[S], os[S];
    float c[2] = {0.f, 0.f};
    if (live) {
      const T* yr = y + row_off(rw.y, (uint32_t)r, rw.seqlen) + c0;
      const T* zr = MODE != kNoGate ? z + row_off(rw.z, (uint32_t)r, rw.seqlen) + c0 : nullptr;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        ys[s].load(yr, s, t, nt, gs);
        os[s].load(dout + r * dim + c0, s, t, nt, gs);
        if (MODE != kNoGate) zs[s].load(zr, s, t, nt, gs);
      }
#pragma unroll
      for (int s = 0; s < S; ++s) {
        float w[kVec], yv[kVec], zv[kVec], go[kVec];
        load_slot<VEC>(weight + c0, s, t, nt, gs, w);
        ys[s].get(yv);
        os[s].get(go);
        if (MODE != kNoGate) zs[s].get(zv);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const float e = MODE != kNoGate ? zv[j] * row::sigmoid<T>(zv[j]) : 1.f;
          const float u = MODE == kNormFirst ? yv[j] : yv[j] * e;
          const float g = MODE == kNormFirst ? go[j] * w[j] * e : go[j] * w[j];
          c[0] = fmaf(u, u, c[0]);
          c[1] = fmaf(g, u, c[1]);
        }
      }
    }
    row::team_sum(c, sums, buf, team, nt);
    buf ^= 1;
    if (!live) continue;
    const float rstd = rsqrtf(c[0] / (float)gs + eps);
    const float k = rstd * rstd * (c[1] / (float)gs);
    T* dzr = MODE != kNoGate ? dz + row_off(rw.dz, (uint32_t)r, rw.seqlen) + c0 : nullptr;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      float w[kVec], yv[kVec], zv[kVec], go[kVec], dyv[kVec], dzv[kVec];
      load_slot<VEC>(weight + c0, s, t, nt, gs, w);
      ys[s].get(yv);
      os[s].get(go);
      if (MODE != kNoGate) zs[s].get(zv);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float sg = MODE != kNoGate ? row::sigmoid<T>(zv[j]) : 1.f;
        const float e = MODE != kNoGate ? zv[j] * sg : 1.f;
        // silu' = sg + z sg (1 - sg); not sg (1 - e) + e, which cancels for large z
        const float de = MODE != kNoGate ? fmaf(e, 1.f - sg, sg) : 0.f;
        const float gw = go[j] * w[j];
        if constexpr (MODE == kNormFirst) {
          const float n = yv[j] * rstd;
          dyv[j] = rstd * fmaf(-yv[j], k, gw * e);
          dzv[j] = gw * n * de;
          dw[s][j] = fmaf(go[j] * e, n, dw[s][j]);
        } else {
          const float u = yv[j] * e;
          const float du = rstd * fmaf(-u, k, gw);
          dyv[j] = du * e;
          dzv[j] = du * yv[j] * de;
          dw[s][j] = fmaf(go[j], u * rstd, dw[s][j]);
        }
      }
      store_slot<VEC>(dy + r * dim + c0, s, t, nt, gs, dyv);
      if (MODE != kNoGate) store_slot<VEC>(dzr, s, t, nt, gs, dzv);
    }
  }
  float* p = part + ((int64_t)blockIdx.x * teams + team) * dim + c0;
#pragma unroll
  for (int s = 0; s < S; ++s) store_slot<VEC>(p, s, t, nt, gs, dw[s]);
}

// ----------------------------------------------------------------- column sum

// 32 columns a CTA, ROWS warps that walk the rows ROWS apart.
template <int ROWS>
__global__ void __launch_bounds__(32 * ROWS)
    column_sum_kernel(const float* __restrict__ part, int64_t rows, int64_t ld, int64_t n,
                      float* __restrict__ out, int64_t n2, float* __restrict__ out2) {
  __shared__ float acc[ROWS][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  const bool in = c < n + n2;
  if (in) {
#pragma unroll 8
    for (int64_t r = w; r < rows; r += ROWS) s += part[r * ld + c];
  }
  acc[w][lane] = s;
  __syncthreads();
  if (w == 0 && in) {
#pragma unroll
    for (int i = 1; i < ROWS; ++i) s += acc[i][lane];
    if (c < n) out[c] = s;
    else out2[c - n] = s;
  }
}

// Slots a thread, by what a kernel holds of each (norm first: the gate too).
// One-element accesses hold every operand unpacked: one slot in the backwards,
// where two would spill (10224 x 2417 in fp32: 291 us).
constexpr int kAddFwdSlots = 4;
constexpr int add_bwd_slots(bool vec) { return vec ? 2 : 1; }
constexpr int gated_fwd_slots(ssd_dtype_t dt, bool norm_first, bool vec) {
  return dt == SSD_DTYPE_BF16 && !norm_first && vec ? 4 : 2;
}
constexpr int gated_bwd_slots(ssd_dtype_t dt, bool vec) {
  return !vec ? 1 : dt == SSD_DTYPE_BF16 ? 4 : 2;
}

// A backward's grid holds the CTAs that its registers let run at once: more
// would be a second, nearly empty round (2560 channels: 366 us instead of 276),
// fewer leave loads out of flight.  Its workspace holds one partial row a team.
constexpr int kAddWarps = 24, kGatedWarps = 32, kManySlotsWarps = 16;   // warps an SM
int64_t bwd_ctas(int64_t rows, const row::Shape& sh, int groups, int warps_of_one_slot) {
  const int warps = sh.slots == 1 ? warps_of_one_slot : kManySlotsWarps;
  const int64_t need = (rows + sh.teams - 1) / sh.teams;
  const int64_t per_sm = std::max(1, warps / (sh.threads() / 32));
  return std::min(need, std::max<int64_t>(1, row::sm_count() * per_sm / groups));
}
int64_t add_bwd_ctas(int64_t rows, const row::Shape& sh, bool vec) {
  return bwd_ctas(rows, sh, 1, vec ? kAddWarps : kManySlotsWarps);
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

int bad(int code, const char* msg) { return set_error(code, msg); }

int launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return SSD_OK;
  char m[256];
  snprintf(m, sizeof(m), "%s launch: %s", what, cudaGetErrorString(e));
  return set_error(SSD_ERR_CUDA, m);
}

bool known(ssd_dtype_t t) { return t == SSD_DTYPE_F32 || t == SSD_DTYPE_BF16; }
size_t esize(ssd_dtype_t t) { return t == SSD_DTYPE_BF16 ? 2 : 4; }
bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_add(int64_t rows, int dim, float eps, ssd_dtype_t dt, ssd_dtype_t rt) {
  if (!known(dt) || !known(rt)) return bad(SSD_ERR_ARG, "unknown dtype");
  if (dt == SSD_DTYPE_F32 && rt != SSD_DTYPE_F32)
    return bad(SSD_ERR_ARG, "an fp32 x takes an fp32 residual");
  if (rows < 1 || dim < 1) return bad(SSD_ERR_ARG, "rows and dim must be >= 1");
  if (rows > 2147483647LL) return bad(SSD_ERR_UNSUPPORTED, "rows must be below 2^31");
  if (dim > row::kMaxRow) return bad(SSD_ERR_UNSUPPORTED, "dim must be at most 16384");
  if (!(eps >= 0.f)) return bad(SSD_ERR_ARG, "eps must be >= 0");
  return SSD_OK;
}

int check_gated(int64_t batch, int64_t seqlen, int dim, int gs, float eps, ssd_dtype_t dt) {
  if (!known(dt)) return bad(SSD_ERR_ARG, "unknown dtype");
  if (batch < 1 || seqlen < 1 || dim < 1 || gs < 1 || dim % gs != 0)
    return bad(SSD_ERR_ARG, "batch, seqlen, dim >= 1 and group_size dividing dim are required");
  if (batch > 2147483647LL || seqlen > 2147483647LL || batch * seqlen > 2147483647LL)
    return bad(SSD_ERR_UNSUPPORTED, "batch * seqlen must be below 2^31");
  if (gs > row::kMaxRow) return bad(SSD_ERR_UNSUPPORTED, "group_size must be at most 16384");
  if (dim / gs > 65535) return bad(SSD_ERR_UNSUPPORTED, "at most 65535 groups");
  if (!(eps >= 0.f)) return bad(SSD_ERR_ARG, "eps must be >= 0");
  return SSD_OK;
}

bool bad_stride(const ssd_stride_t& s) {
  return s.batch < 0 || s.token < 0 || s.batch > (1LL << 40) || s.token > (1LL << 40);
}
// all rows of [batch, seqlen] one stride apart
bool even(const ssd_stride_t& s, int64_t batch, int64_t seqlen) {
  return batch == 1 || s.batch == seqlen * s.token;
}
bool wide_stride(const ssd_stride_t& s, size_t e) {
  return (s.batch * (int64_t)e) % 16 == 0 && (s.token * (int64_t)e) % 16 == 0;
}

}  // namespace norm

void launch_column_sum(const float* part, int64_t rows, int64_t ld, int64_t n, float* out,
                       int64_t n2, float* out2, cudaStream_t st) {
  // many rows: more of them at once (1024 rows of 1280 columns: 22 us with 8
  // warps, whose loads wait for one another)
  const unsigned grid = (unsigned)((n + n2 + 31) / 32);
  if (rows >= 128)
    norm::column_sum_kernel<32><<<grid, 1024, 0, st>>>(part, rows, ld, n, out, n2, out2);
  else
    norm::column_sum_kernel<8><<<grid, 256, 0, st>>>(part, rows, ld, n, out, n2, out2);
}

}  // namespace ssd

using namespace ssd;
using namespace ssd::norm;

// Launches the wide or one-element instance with the shape's slots.
#define SSD_NORM_SLOTS(LAUNCH, V)    \
  switch (sh.slots) {                \
    case 1: LAUNCH(V, 1); break;     \
    case 2: LAUNCH(V, 2); break;     \
    case 3: LAUNCH(V, 3); break;     \
    default: LAUNCH(V, 4); break;    \
  }
#define SSD_GATED_MODE(LAUNCH, T, V, S)                      \
  do {                                                       \
    if (!z) LAUNCH(T, V, S, kNoGate);                        \
    else if (norm_before_gate) LAUNCH(T, V, S, kNormFirst);  \
    else LAUNCH(T, V, S, kGateFirst);                        \
  } while (0)
#define SSD_NORM_PICK(LAUNCH)              \
  do {                                     \
    if (vec) SSD_NORM_SLOTS(LAUNCH, true)  \
    else SSD_NORM_SLOTS(LAUNCH, false)     \
  } while (0)

extern "C" {

int ssd_block_abi_version(void) { return SSD_BLOCK_ABI_VERSION; }

int ssd_add_rmsnorm_fwd(const void* x, const void* residual, const float* scale,
                        const float* weight, float eps, int64_t rows, int dim, ssd_dtype_t dtype,
                        ssd_dtype_t residual_dtype, void* y, void* residual_out, void* stream) {
  const int c = check_add(rows, dim, eps, dtype, residual_dtype);
  if (c != SSD_OK) return c;
  if (!x || !weight || !y || !residual_out)
    return bad(SSD_ERR_NULL, "x, weight, y and residual_out are required");
  const size_t e = esize(dtype), re = esize(residual_dtype);
  if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(residual, re) ||
      !aligned_to(residual_out, re) || !aligned_to(weight, 4) || !aligned_to(scale, 4))
    return bad(SSD_ERR_ALIGN, "a pointer is not aligned to its element");
  const bool vec = dim % kVec == 0 && row::wide(x) && row::wide(residual) && row::wide(y) &&
                   row::wide(residual_out) && row::wide(scale) && row::wide(weight);
  const row::Shape sh = row::shape_for(dim, kAddFwdSlots);
  const unsigned grid = (unsigned)((rows + sh.teams - 1) / sh.teams);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  using bf = __nv_bfloat16;
#define SSD_ADD_FWD(T, R, V, S)                                                              \
  add_fwd_kernel<T, R, V, S><<<grid, sh.threads(), 0, st>>>(                                 \
      static_cast<const T*>(x), static_cast<const R*>(residual), scale, weight, eps,         \
      (uint32_t)rows, dim, sh.nt, static_cast<T*>(y), static_cast<R*>(residual_out))
#define SSD_ADD_FWD_FF(V, S) SSD_ADD_FWD(float, float, V, S)
#define SSD_ADD_FWD_BF(V, S) SSD_ADD_FWD(bf, float, V, S)
#define SSD_ADD_FWD_BB(V, S) SSD_ADD_FWD(bf, bf, V, S)
  if (dtype == SSD_DTYPE_F32) SSD_NORM_PICK(SSD_ADD_FWD_FF);
  else if (residual_dtype == SSD_DTYPE_F32) SSD_NORM_PICK(SSD_ADD_FWD_BF);
  else SSD_NORM_PICK(SSD_ADD_FWD_BB);
  return launched("add_rmsnorm_fwd");
}

size_t ssd_add_rmsnorm_bwd_workspace_bytes(int64_t rows, int dim) {
  if (check_add(rows, dim, 0.f, SSD_DTYPE_F32, SSD_DTYPE_F32) != SSD_OK) return 0;
  int64_t most = 0;   // of the layouts for aligned rows and others
  for (const bool vec : {false, true}) {
    const row::Shape sh = row::shape_for(dim, add_bwd_slots(vec));
    most = std::max(most, add_bwd_ctas(rows, sh, vec) * sh.teams);
  }
  return up256((size_t)most * 2 * dim * sizeof(float));
}

int ssd_add_rmsnorm_bwd(const void* dy, const void* dresidual_out, const void* residual_out,
                        const void* x, const float* scale, const float* weight, float eps,
                        int64_t rows, int dim, ssd_dtype_t dtype, ssd_dtype_t residual_dtype,
                        void* dx, void* dresidual, float* dweight, float* dscale, void* workspace,
                        size_t workspace_bytes, void* stream) {
  const int c = check_add(rows, dim, eps, dtype, residual_dtype);
  if (c != SSD_OK) return c;
  if (!dy || !residual_out || !weight || !dweight || !workspace)
    return bad(SSD_ERR_NULL, "dy, residual_out, weight, dweight and workspace are required");
  if ((scale != nullptr) != (dscale != nullptr) || (scale && !x))
    return bad(SSD_ERR_NULL, "scale takes x and dscale, and dscale takes scale");
  const size_t e = esize(dtype), re = esize(residual_dtype);
  if (!aligned_to(dy, e) || !aligned_to(x, e) || !aligned_to(dx, e) ||
      !aligned_to(dresidual_out, re) || !aligned_to(residual_out, re) ||
      !aligned_to(dresidual, re) || !aligned_to(weight, 4) || !aligned_to(scale, 4) ||
      !aligned_to(dweight, 4) || !aligned_to(dscale, 4))
    return bad(SSD_ERR_ALIGN, "a pointer is not aligned to its element");
  if (!aligned_to(workspace, 256)) return bad(SSD_ERR_ALIGN, "workspace: 256-byte aligned");
  if (workspace_bytes < ssd_add_rmsnorm_bwd_workspace_bytes(rows, dim))
    return bad(SSD_ERR_WORKSPACE, "workspace too small");
  const bool vec = dim % kVec == 0 && row::wide(dy) && row::wide(dresidual_out) &&
                   row::wide(residual_out) && row::wide(x) && row::wide(dx) &&
                   row::wide(dresidual) && row::wide(scale) && row::wide(weight);
  const row::Shape sh = row::shape_for(dim, add_bwd_slots(vec));
  const unsigned grid = (unsigned)add_bwd_ctas(rows, sh, vec);
  float* part = static_cast<float*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  using bf = __nv_bfloat16;
#define SSD_ADD_BWD(T, R, V, S)                                                               \
  add_bwd_kernel<T, R, V, S><<<grid, sh.threads(), 0, st>>>(                                  \
      static_cast<const T*>(dy), static_cast<const R*>(dresidual_out),                        \
      static_cast<const R*>(residual_out), static_cast<const T*>(x), scale, weight, eps,      \
      (uint32_t)rows, dim, sh.nt, static_cast<T*>(dx), static_cast<R*>(dresidual), part)
#define SSD_ADD_BWD_FF(V, S) SSD_ADD_BWD(float, float, V, S)
#define SSD_ADD_BWD_BF(V, S) SSD_ADD_BWD(bf, float, V, S)
#define SSD_ADD_BWD_BB(V, S) SSD_ADD_BWD(bf, bf, V, S)
  if (dtype == SSD_DTYPE_F32) SSD_NORM_PICK(SSD_ADD_BWD_FF);
  else if (residual_dtype == SSD_DTYPE_F32) SSD_NORM_PICK(SSD_ADD_BWD_BF);
  else SSD_NORM_PICK(SSD_ADD_BWD_BB);
  const int64_t prow = (int64_t)grid * sh.teams;
  launch_column_sum(part, prow, 2 * dim, dim, dweight, dscale ? dim : 0, dscale, st);
  return launched("add_rmsnorm_bwd");
}

int ssd_gated_rmsnorm_fwd(const void* y, ssd_stride_t y_stride, const void* z,
                          ssd_stride_t z_stride, const float* weight, float eps, int64_t batch,
                          int64_t seqlen, int dim, int group_size, int norm_before_gate,
                          ssd_dtype_t dtype, void* out, void* stream) {
  const int c = check_gated(batch, seqlen, dim, group_size, eps, dtype);
  if (c != SSD_OK) return c;
  if (!y || !weight || !out) return bad(SSD_ERR_NULL, "y, weight and out are required");
  const size_t e = esize(dtype);
  if (!aligned_to(y, e) || !aligned_to(z, e) || !aligned_to(out, e) || !aligned_to(weight, 4))
    return bad(SSD_ERR_ALIGN, "a pointer is not aligned to its element");
  if (bad_stride(y_stride) || (z && bad_stride(z_stride)))
    return bad(SSD_ERR_ARG, "strides must be in [0, 2^40]");
  const bool vec = group_size % kVec == 0 && row::wide(y) && row::wide(z) && row::wide(out) &&
                   row::wide(weight) && wide_stride(y_stride, e) &&
                   (!z || wide_stride(z_stride, e));
  const row::Shape sh = row::shape_for(group_size, gated_fwd_slots(dtype, z && norm_before_gate, vec));
  Rows rw = {(uint32_t)(batch * seqlen), (uint32_t)seqlen, {y_stride.batch, y_stride.token},
             {z_stride.batch, z_stride.token}, {0, 0}};
  if (even(y_stride, batch, seqlen) && (!z || even(z_stride, batch, seqlen))) rw.seqlen = 0;
  const dim3 grid((unsigned)((rw.rows + (int64_t)sh.teams - 1) / sh.teams),
                  (unsigned)(dim / group_size));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
#define SSD_GATED_FWD(T, V, S, MODE)                                                       \
  gated_fwd_kernel<T, V, S, MODE><<<grid, sh.threads(), 0, st>>>(                          \
      static_cast<const T*>(y), static_cast<const T*>(z), weight, eps, rw, dim, group_size, \
      sh.nt, static_cast<T*>(out))
#define SSD_GATED_FWD_F(V, S) SSD_GATED_MODE(SSD_GATED_FWD, float, V, S)
#define SSD_GATED_FWD_B(V, S) SSD_GATED_MODE(SSD_GATED_FWD, __nv_bfloat16, V, S)
  if (dtype == SSD_DTYPE_F32) SSD_NORM_PICK(SSD_GATED_FWD_F);
  else SSD_NORM_PICK(SSD_GATED_FWD_B);
  return launched("gated_rmsnorm_fwd");
}

size_t ssd_gated_rmsnorm_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int dim,
                                             int group_size) {
  if (check_gated(batch, seqlen, dim, group_size, 0.f, SSD_DTYPE_F32) != SSD_OK) return 0;
  size_t most = 0;   // of the layouts for one slot, two and four
  for (int i = 0; i < 3; ++i) {
    const ssd_dtype_t dt = i == 2 ? SSD_DTYPE_BF16 : SSD_DTYPE_F32;
    const row::Shape sh = row::shape_for(group_size, gated_bwd_slots(dt, i > 0));
    most = std::max(most, (size_t)(bwd_ctas(batch * seqlen, sh, dim / group_size, kGatedWarps) * sh.teams));
  }
  return up256(most * dim * sizeof(float));
}

int ssd_gated_rmsnorm_bwd(const void* dout, const void* y, ssd_stride_t y_stride, const void* z,
                          ssd_stride_t z_stride, const float* weight, float eps, int64_t batch,
                          int64_t seqlen, int dim, int group_size, int norm_before_gate,
                          ssd_dtype_t dtype, void* dy, void* dz, ssd_stride_t dz_stride,
                          float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
  const int c = check_gated(batch, seqlen, dim, group_size, eps, dtype);
  if (c != SSD_OK) return c;
  if (!dout || !y || !weight || !dy || !dweight || !workspace)
    return bad(SSD_ERR_NULL, "dout, y, weight, dy, dweight and workspace are required");
  if ((z != nullptr) != (dz != nullptr)) return bad(SSD_ERR_NULL, "z and dz come together");
  const size_t e = esize(dtype);
  if (!aligned_to(dout, e) || !aligned_to(y, e) || !aligned_to(z, e) || !aligned_to(dy, e) ||
      !aligned_to(dz, e) || !aligned_to(weight, 4) || !aligned_to(dweight, 4))
    return bad(SSD_ERR_ALIGN, "a pointer is not aligned to its element");
  if (!aligned_to(workspace, 256)) return bad(SSD_ERR_ALIGN, "workspace: 256-byte aligned");
  if (bad_stride(y_stride) || (z && (bad_stride(z_stride) || bad_stride(dz_stride))))
    return bad(SSD_ERR_ARG, "strides must be in [0, 2^40]");
  if (z && ((seqlen > 1 && dz_stride.token < dim) || (batch > 1 && dz_stride.batch < dim)))
    return bad(SSD_ERR_ARG, "dz: tokens must not overlap");
  if (workspace_bytes < ssd_gated_rmsnorm_bwd_workspace_bytes(batch, seqlen, dim, group_size))
    return bad(SSD_ERR_WORKSPACE, "workspace too small");
  const bool vec = group_size % kVec == 0 && row::wide(dout) && row::wide(y) && row::wide(z) &&
                   row::wide(dy) && row::wide(dz) && row::wide(weight) &&
                   wide_stride(y_stride, e) &&
                   (!z || (wide_stride(z_stride, e) && wide_stride(dz_stride, e)));
  const row::Shape sh = row::shape_for(group_size, gated_bwd_slots(dtype, vec));
  Rows rw = {(uint32_t)(batch * seqlen), (uint32_t)seqlen, {y_stride.batch, y_stride.token},
             {z_stride.batch, z_stride.token}, {dz_stride.batch, dz_stride.token}};
  if (even(y_stride, batch, seqlen) &&
      (!z || (even(z_stride, batch, seqlen) && even(dz_stride, batch, seqlen))))
    rw.seqlen = 0;
  const dim3 grid((unsigned)bwd_ctas(rw.rows, sh, dim / group_size, kGatedWarps),
                  (unsigned)(dim / group_size));
  float* part = static_cast<float*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
#define SSD_GATED_BWD(T, V, S, MODE)                                                          \
  gated_bwd_kernel<T, V, S, MODE><<<grid, sh.threads(), 0, st>>>(                             \
      static_cast<const T*>(dout), static_cast<const T*>(y), static_cast<const T*>(z), weight, \
      eps, rw, dim, group_size, sh.nt, static_cast<T*>(dy), static_cast<T*>(dz), part)
#define SSD_GATED_BWD_F(V, S) SSD_GATED_MODE(SSD_GATED_BWD, float, V, S)
#define SSD_GATED_BWD_B(V, S) SSD_GATED_MODE(SSD_GATED_BWD, __nv_bfloat16, V, S)
  if (dtype == SSD_DTYPE_F32) SSD_NORM_PICK(SSD_GATED_BWD_F);
  else SSD_NORM_PICK(SSD_GATED_BWD_B);
  launch_column_sum(part, (int64_t)grid.x * sh.teams, dim, dim, dweight, 0, nullptr, st);
  return launched("gated_rmsnorm_bwd");
}

}  // extern "C"
