// The global 2-norm of a set of gradients and their clipping by it:
//   norm = sqrt(sum over all tensors of g^2),
//   out  = g * min(1, max_norm / (norm + eps))
// Bound by HBM: the norm reads every gradient once; clipping reads it once
// more and writes it (nothing, where the norm is below max_norm and the
// gradients stay in place).  The second pass walks the tensors backwards, so
// that what the first pass left in the L2 cache is read from there.
//
// The tensors come as a table in the kernel's parameters (no copy to the
// device, capturable as is), cut into chunks that CTAs take a grid apart.
// Squares are summed in fp32 over at most kChunk / kThreads values, then in
// double: per thread over its chunks, over the CTA, and over the CTAs'
// partial sums, always in the same order.  Values whose squares leave the
// fp32 range are squared in double.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>

#include "../../include/ssd_block.h"
#include "ssd_common.cuh"
#include "ssd_row.cuh"

namespace ssd {
namespace clip {

constexpr int kThreads = 256;
constexpr int kChunk = 16384;      // elements
// CTAs an SM: reading alone wants all the loads that fit, reading and writing
// together fewer (645M bf16 values into fp32: 634 us with 5, 776 with 8, 700
// with 4; stores that leave the L2 first were no faster).
constexpr int kNormCtas = 8, kScaleCtas = 5;
constexpr int kSmall = 48, kLarge = 768;   // tensors a launch: 1.5 KB or 23 KB of parameters

template <int N>
struct Table {
  const void* g[N];
  void* out[N];          // null: nothing to write (norm only)
  int64_t n[N];
  uint32_t first[N];     // the tensor's first chunk in this launch
  uint8_t g_bf16[N], out_bf16[N];
  uint32_t tensors, chunks;
};

template <int N>
__device__ __forceinline__ uint32_t tensor_of(const Table<N>& t, uint32_t chunk) {
  uint32_t lo = 0, hi = t.tensors;   // the last tensor whose first chunk is <= chunk
  while (hi - lo > 1) {
    const uint32_t m = (lo + hi) / 2;
    if (t.first[m] <= chunk) lo = m;
    else hi = m;
  }
  return lo;
}

// Elements before the first 16-byte boundary.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int n) {
  const int h = (int)(((16 - ((uintptr_t)p & 15)) & 15) / sizeof(T));
  return h < n ? h : n;
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s += part[i];
  return s;
}

struct SquareSum {
  float f = 0.f;    // of the current chunk
  double d = 0.0;
  // Eight values at once.  Their fp32 sum is taken where it is neither too large
  // nor so small that squares lost to underflow could matter to it.
  __device__ __forceinline__ void add8(const float (&v)[row::kVec]) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < row::kVec; ++j) s = fmaf(v[j], v[j], s);
    if (s >= 0x1p-80f && s < 0x1p120f) {
      f += s;
    } else {
      float big = 0.f;
#pragma unroll
      for (int j = 0; j < row::kVec; ++j) big = fmaxf(big, fabsf(v[j]));
      if (s != 0.f || big != 0.f) {   // (a NaN is in s)
#pragma unroll
        for (int j = 0; j < row::kVec; ++j) d += (double)v[j] * (double)v[j];
      }
    }
  }
  __device__ __forceinline__ void add1(float v) { d += (double)v * (double)v; }
  __device__ __forceinline__ void flush() {
    d += f;
    f = 0.f;
  }
};

__device__ __forceinline__ void load8(const float* p, float (&v)[row::kVec]) {
  row::load_slot<true>(p, 0, 0, 1, row::kVec, v);
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[row::kVec]) {
  row::load_slot<true>(p, 0, 0, 1, row::kVec, v);
}

template <typename T>
__device__ __forceinline__ void square_chunk(const T* p, int n, SquareSum& acc) {
  const int head = head_of(p, n);
  if ((int)threadIdx.x < head) acc.add1(to_f(p[threadIdx.x]));
  const T* q = p + head;
  const int vecs = (n - head) / row::kVec;
#pragma unroll 4
  for (int i = threadIdx.x; i < vecs; i += kThreads) {
    float v[row::kVec];
    load8(q + i * row::kVec, v);
    acc.add8(v);
  }
  const int rest = head + vecs * row::kVec + threadIdx.x;
  if (rest < n) acc.add1(to_f(p[rest]));
  acc.flush();
}

template <int N>
__global__ void __launch_bounds__(kThreads)
    square_sum_kernel(const __grid_constant__ Table<N> t, double* __restrict__ part) {
  SquareSum acc;
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const uint32_t k = tensor_of(t, c);
    const int64_t at = (int64_t)(c - t.first[k]) * kChunk;
    const int64_t left = t.n[k] - at;
    const int n = (int)(left < kChunk ? left : kChunk);
    if (t.g_bf16[k]) square_chunk(static_cast<const __nv_bfloat16*>(t.g[k]) + at, n, acc);
    else square_chunk(static_cast<const float*>(t.g[k]) + at, n, acc);
  }
  const double s = block_sum(acc.d);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// sqrt of the partial sums' total, in every thread; the same order in every CTA.
__device__ __forceinline__ double norm_of(const double* __restrict__ part, int parts) {
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) s += part[i];
  return sqrt(block_sum(s));
}

__global__ void __launch_bounds__(kThreads)
    norm_kernel(const double* __restrict__ part, int parts, float* __restrict__ norm) {
  const double v = norm_of(part, parts);
  if (threadIdx.x == 0) *norm = (float)v;
}

// (g and o may be the same memory: each element is read and written by one thread)
// The factor is first * coef: first is 1, or 2^-64 where the factor alone would be
// a subnormal of few bits.
template <typename T, typename O>
__device__ __forceinline__ void scale_chunk(const T* p, O* o, int n, float first, float coef) {
  const int head = head_of(p, n);
  if ((int)threadIdx.x < head) o[threadIdx.x] = from_f<O>(to_f(p[threadIdx.x]) * first * coef);
  const int vecs = (n - head) / row::kVec;
  const bool wide = ((uintptr_t)(o + head) & 15) == 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < vecs; i += kThreads) {
    float v[row::kVec];
    load8(p + head + i * row::kVec, v);
#pragma unroll
    for (int j = 0; j < row::kVec; ++j) v[j] = v[j] * first * coef;
    O* at = o + head + i * row::kVec;
    if (wide) {
      row::store_slot<true>(at, 0, 0, 1, row::kVec, v);
    } else {
#pragma unroll
      for (int j = 0; j < row::kVec; ++j) at[j] = from_f<O>(v[j]);
    }
  }
  const int rest = head + vecs * row::kVec + threadIdx.x;
  if (rest < n) o[rest] = from_f<O>(to_f(p[rest]) * first * coef);
}

template <int N>
__global__ void __launch_bounds__(kThreads)
    scale_kernel(const __grid_constant__ Table<N> t, const double* __restrict__ part, int parts,
                 float max_norm, float eps, int in_place, float* __restrict__ norm) {
  using bf = __nv_bfloat16;
  const double v = norm_of(part, parts);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)v;
  // a NaN norm compares false and is kept
  const double c = (double)max_norm / (v + (double)eps);
  const bool tiny = c < 0x1p-100;
  const float first = tiny ? 0x1p-64f : 1.f;
  const float coef = c >= 1.0 ? 1.f : (float)(tiny ? c * 0x1p64 : c);
  if (in_place && coef == 1.f) return;
  for (uint32_t i = blockIdx.x; i < t.chunks; i += gridDim.x) {
    const uint32_t ch = t.chunks - 1 - i;
    const uint32_t k = tensor_of(t, ch);
    const int64_t at = (int64_t)(ch - t.first[k]) * kChunk;
    const int64_t left = t.n[k] - at;
    const int n = (int)(left < kChunk ? left : kChunk);
    if (t.g_bf16[k]) {
      const bf* p = static_cast<const bf*>(t.g[k]) + at;
      if (t.out_bf16[k]) scale_chunk(p, static_cast<bf*>(t.out[k]) + at, n, first, coef);
      else scale_chunk(p, static_cast<float*>(t.out[k]) + at, n, first, coef);
    } else {
      const float* p = static_cast<const float*>(t.g[k]) + at;
      if (t.out_bf16[k]) scale_chunk(p, static_cast<bf*>(t.out[k]) + at, n, first, coef);
      else scale_chunk(p, static_cast<float*>(t.out[k]) + at, n, first, coef);
    }
  }
}

int bad(int code, const char* msg) { return set_error(code, msg); }

int grid_of(uint32_t chunks, int ctas_per_sm) {
  return (int)std::min<int64_t>(chunks, (int64_t)row::sm_count() * ctas_per_sm);
}

// Fills the next launch's table from tensor `k` on; returns the tensor after
// it.  Empty tensors are left out.
template <int N>
int fill(Table<N>& t, int k, int count, const void* const* g, const int64_t* n,
         const int32_t* gt, void* const* out, const int32_t* ot) {
  t.tensors = t.chunks = 0;
  for (; k < count && t.tensors < N; ++k) {
    if (n[k] == 0) continue;
    const int64_t chunks = (n[k] + kChunk - 1) / kChunk;
    if (t.tensors > 0 && t.chunks + chunks > 0x7fffffff) break;
    const uint32_t i = t.tensors++;
    t.g[i] = g[k];
    t.out[i] = out ? out[k] : nullptr;
    t.n[i] = n[k];
    t.first[i] = t.chunks;
    t.g_bf16[i] = gt[k] == SSD_DTYPE_BF16;
    t.out_bf16[i] = out && (ot ? ot[k] : gt[k]) == SSD_DTYPE_BF16;
    t.chunks += (uint32_t)chunks;
  }
  return k;
}

template <int N>
int run(const void* const* g, const int64_t* n, const int32_t* gt, int count, void* const* out,
        const int32_t* ot, bool clipping, float max_norm, float eps, float* norm, double* part,
        cudaStream_t st) {
  static thread_local Table<N> t;   // too large for some callers' stacks
  const bool in_place = clipping && !out;
  void* const* to = out ? out : const_cast<void* const*>(g);
  int parts = 0;
  for (int k = 0; k < count;) {
    k = fill(t, k, count, g, n, gt, clipping ? to : nullptr, out ? ot : nullptr);
    if (t.chunks == 0) break;
    const int grid = grid_of(t.chunks, kNormCtas);
    square_sum_kernel<N><<<grid, kThreads, 0, st>>>(t, part + parts);
    parts += grid;
  }
  if (!clipping || parts == 0) {
    norm_kernel<<<1, kThreads, 0, st>>>(part, parts, norm);
  } else {
    bool first = true;
    for (int k = 0; k < count;) {
      k = fill(t, k, count, g, n, gt, to, out ? ot : nullptr);
      if (t.chunks == 0) break;
      scale_kernel<N><<<grid_of(t.chunks, kScaleCtas), kThreads, 0, st>>>(t, part, parts, max_norm, eps,
                                                              in_place, first ? norm : nullptr);
      first = false;
    }
  }
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return SSD_OK;
  char m[256];
  snprintf(m, sizeof(m), "clip_grads launch: %s", cudaGetErrorString(e));
  return set_error(SSD_ERR_CUDA, m);
}

int check(const void* const* g, const int64_t* n, const int32_t* gt, int count, void* const* out,
          const int32_t* ot, const float* norm, const void* ws, size_t ws_bytes) {
  if (count < 0) return bad(SSD_ERR_ARG, "count must be >= 0");
  if (count > 0 && (!g || !n || !gt)) return bad(SSD_ERR_NULL, "grads, sizes and dtypes are required");
  if (!norm || !ws) return bad(SSD_ERR_NULL, "norm and workspace are required");
  if (((uintptr_t)norm & 3) || ((uintptr_t)ws & 255))
    return bad(SSD_ERR_ALIGN, "norm must be 4-byte, workspace 256-byte aligned");
  for (int k = 0; k < count; ++k) {
    if (n[k] < 0) return bad(SSD_ERR_ARG, "sizes must be >= 0");
    if (n[k] > (1LL << 44)) return bad(SSD_ERR_UNSUPPORTED, "a size is above 2^44");
    if (n[k] == 0) continue;
    const int32_t o = ot ? ot[k] : gt[k];
    if ((gt[k] != SSD_DTYPE_F32 && gt[k] != SSD_DTYPE_BF16) ||
        (o != SSD_DTYPE_F32 && o != SSD_DTYPE_BF16))
      return bad(SSD_ERR_ARG, "unknown dtype");
    if (!g[k] || (out && !out[k])) return bad(SSD_ERR_NULL, "a gradient or output is NULL");
    if (((uintptr_t)g[k] & (gt[k] == SSD_DTYPE_BF16 ? 1 : 3)) ||
        (out && ((uintptr_t)out[k] & (o == SSD_DTYPE_BF16 ? 1 : 3))))
      return bad(SSD_ERR_ALIGN, "a pointer is not aligned to its element");
  }
  if (ws_bytes < ssd_clip_grads_workspace_bytes(count))
    return bad(SSD_ERR_WORKSPACE, "workspace too small");
  return SSD_OK;
}

}  // namespace clip
}  // namespace ssd

using namespace ssd::clip;

extern "C" {

size_t ssd_clip_grads_workspace_bytes(int count) {
  if (count < 0) return 0;
  // one double per CTA of each launch
  const size_t launches = (size_t)count / kSmall + 1;
  return (launches * ssd::row::sm_count() * kNormCtas * sizeof(double) + 255) & ~(size_t)255;
}

int ssd_grad_norm(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int count,
                  float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  const int c = check(grads, sizes, dtypes, count, nullptr, nullptr, norm, workspace,
                      workspace_bytes);
  if (c != SSD_OK) return c;
  double* part = static_cast<double*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return count <= kSmall ? run<kSmall>(grads, sizes, dtypes, count, nullptr, nullptr, false, 0.f,
                                       0.f, norm, part, st)
                         : run<kLarge>(grads, sizes, dtypes, count, nullptr, nullptr, false, 0.f,
                                       0.f, norm, part, st);
}

int ssd_clip_grads(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int count,
                   void* const* outs, const int32_t* out_dtypes, float max_norm, float eps,
                   float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  const int c = check(grads, sizes, dtypes, count, outs, outs ? out_dtypes : nullptr, norm,
                      workspace, workspace_bytes);
  if (c != SSD_OK) return c;
  if (!(max_norm >= 0.f) || !(eps >= 0.f)) return bad(SSD_ERR_ARG, "max_norm and eps must be >= 0");
  double* part = static_cast<double*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return count <= kSmall ? run<kSmall>(grads, sizes, dtypes, count, outs, out_dtypes, true,
                                       max_norm, eps, norm, part, st)
                         : run<kLarge>(grads, sizes, dtypes, count, outs, out_dtypes, true,
                                       max_norm, eps, norm, part, st);
}

}  // extern "C"
