// Helpers shared by the row-wise kernels of the block's operators: a team of
// warps that holds one row (or one channel group of a row) in registers,
// eight elements to a slot, and the sum over the rows of partial parameter
// gradients.
#pragma once

#include "ssd_common.cuh"

namespace ssd {
namespace row {

constexpr int kVec = 8;   // elements per slot: one 16-byte bf16 or two fp32 vectors
constexpr int kMaxWarps = 16;   // of a CTA of row teams

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The sigmoid for data of type T.  bf16: 1 / (1 + 2^(-v log2 e)) in four
// instructions, each SFU operation within about 2^-22 and the rounded exponent
// adding |v| 2^-24, which is nothing beside bf16's 2^-9 (with expf and a division
// the gated backward was bound by its instructions).  fp32: expf, whose error does
// not grow with v; its calls move twice the bytes for the same instructions.
// Subnormals flush, where the sigmoid is 0 to fp32's normal range.
template <typename T>
__device__ __forceinline__ float sigmoid(float v) {
  if constexpr (sizeof(T) == 2) return rcp(1.f + ex2(-kLog2e * v));
  else return rcp(1.f + expf(-v));
}

__device__ __forceinline__ void unpack(uint4 w, float (&v)[kVec]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

// Column of element j of slot s for thread t of a team of nt.  VEC: a slot is
// eight consecutive columns (one wide access); otherwise a slot's elements are
// nt apart, so that the team's one-element accesses are consecutive.
template <bool VEC>
__device__ __forceinline__ int col_of(int s, int j, int t, int nt) {
  return VEC ? (s * nt + t) * kVec + j : (s * kVec + j) * nt + t;
}

// Slot s of a row of n elements; zeros past n (n is a multiple of 8 if VEC).
template <bool VEC>
__device__ __forceinline__ void load_slot(const float* p, int s, int t, int nt, int n,
                                          float (&v)[kVec]) {
  if constexpr (VEC) {
    const int c = col_of<true>(s, 0, t, nt);
    if (c < n) {
      const float4 a = *reinterpret_cast<const float4*>(p + c);
      const float4 b = *reinterpret_cast<const float4*>(p + c + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[j] = 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int c = col_of<false>(s, j, t, nt);
      v[j] = c < n ? p[c] : 0.f;
    }
  }
}
template <bool VEC>
__device__ __forceinline__ void load_slot(const __nv_bfloat16* p, int s, int t, int nt, int n,
                                          float (&v)[kVec]) {
  if constexpr (VEC) {
    const int c = col_of<true>(s, 0, t, nt);
    unpack(c < n ? *reinterpret_cast<const uint4*>(p + c) : make_uint4(0, 0, 0, 0), v);
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int c = col_of<false>(s, j, t, nt);
      v[j] = c < n ? __bfloat162float(p[c]) : 0.f;
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void store_slot(float* p, int s, int t, int nt, int n,
                                           const float (&v)[kVec]) {
  if constexpr (VEC) {
    const int c = col_of<true>(s, 0, t, nt);
    if (c < n) {
      *reinterpret_cast<float4*>(p + c) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(p + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int c = col_of<false>(s, j, t, nt);
      if (c < n) p[c] = v[j];
    }
  }
}
template <bool VEC>
__device__ __forceinline__ void store_slot(__nv_bfloat16* p, int s, int t, int nt, int n,
                                           const float (&v)[kVec]) {
  if constexpr (VEC) {
    const int c = col_of<true>(s, 0, t, nt);
    if (c < n) {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(p + c) = make_uint4(u[0], u[1], u[2], u[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int c = col_of<false>(s, j, t, nt);
      if (c < n) p[c] = __float2bfloat16_rn(v[j]);
    }
  }
}

// The value as it is stored in type T.
__device__ __forceinline__ float stored(float v, const float*) { return v; }
__device__ __forceinline__ float stored(float v, const __nv_bfloat16*) {
  return __bfloat162float(__float2bfloat16_rn(v));
}

// A slot as it was loaded: bf16 stays packed (four registers) until its values
// are used, so that a thread can hold several rows' operands at once.
template <typename T, bool VEC>
struct Slot {
  float v[kVec];
  __device__ __forceinline__ void load(const T* p, int s, int t, int nt, int n) {
    load_slot<VEC>(p, s, t, nt, n, v);
  }
  __device__ __forceinline__ void get(float (&o)[kVec]) const {
#pragma unroll
    for (int j = 0; j < kVec; ++j) o[j] = v[j];
  }
};
template <>
struct Slot<__nv_bfloat16, true> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int s, int t, int nt, int n) {
    const int c = col_of<true>(s, 0, t, nt);
    u = c < n ? *reinterpret_cast<const uint4*>(p + c) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&o)[kVec]) const { unpack(u, o); }
};

// Sums of K values over a team of nt consecutive threads (8, 16 or whole
// warps; team `team` of the CTA), to every thread of it.  Every thread of the
// CTA calls it the same number of times; `buf` alternates between 0 and 1 from
// call to call, so that one barrier a call is enough: a slow reader of one
// call's sums is past the next call's barrier before their place is written
// again.
struct TeamSums {
  float part[2][2][kMaxWarps];
};
template <int K>
__device__ __forceinline__ void team_sum(float (&a)[K], TeamSums& sm, int buf, int team, int nt) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    if (off < nt) {
#pragma unroll
      for (int k = 0; k < K; ++k) a[k] += __shfl_xor_sync(0xffffffffu, a[k], off);
    }
  if (nt <= 32) return;
  const int warp = threadIdx.x >> 5, warps = nt >> 5;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) sm.part[buf][k][warp] = a[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) a[k] = 0.f;
  for (int i = 0; i < warps; ++i)
#pragma unroll
    for (int k = 0; k < K; ++k) a[k] += sm.part[buf][k][team * warps + i];
}

// How a row of n elements is laid over threads: nt threads a row (8, 16 or
// whole warps) with `slots` slots of eight elements each, `teams` rows at once
// in a CTA.  Among up to `most` slots a thread the fullest threads are taken,
// and then the fewest, whose sums cost least to exchange; four slots where
// sixteen warps need them.
constexpr int kMaxRow = 16384, kRowThreads = 512, kTeamThreads = 256;
struct Shape {
  int nt, slots, teams;
  int threads() const { return nt * teams; }
};
inline Shape shape_for(int n, int most) {
  const int vecs = (n + kVec - 1) / kVec;
  if (vecs > kRowThreads * most) most = 4;   // n <= kMaxRow
  Shape s = {0, 0, 0};
  for (int k = 1; k <= most; ++k) {
    const int need = (vecs + k - 1) / k;
    const int nt = need <= 8 ? 8 : need <= 16 ? 16 : (need + 31) / 32 * 32;
    if (nt <= kRowThreads && (s.nt == 0 || nt * k <= s.nt * s.slots)) {
      s.nt = nt;
      s.slots = k;
    }
  }
  s.teams = s.nt >= kTeamThreads ? 1 : kTeamThreads / s.nt;
  return s;
}

inline bool wide(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int sm_count();

}  // namespace row

// Column sums in a fixed order: s[c] = sum over r < rows of part[r * ld + c] for
// c < n + n2; the first n go to out, the next n2 to out2.  Its launch error and
// those before it are left to the caller's cudaGetLastError.
void launch_column_sum(const float* part, int64_t rows, int64_t ld, int64_t n, float* out,
                       int64_t n2, float* out2, cudaStream_t st);

}  // namespace ssd
