// What the gated delta rule's two passes along the sequence share: a warp with 16
// rows of a state in registers, its products and its results' way to memory.
#pragma once

#include "ssd_delta.cuh"

namespace ssd {
namespace delta {

// Warps of a CTA that have rows of the state (at most), and those that only load: rows
// have to be split into terms on their way, which took the former's time otherwise.
constexpr int kRowWarps = 4, kLoadWarps = 4;

__device__ __forceinline__ float2 ld2(const float* p) { return *reinterpret_cast<const float2*>(p); }

// d += a B^T for lower triangular B [i][j] in shared memory: a [.., j] as term
// operands of 16 columns, d [.., i].
template <int C, int NT>
__device__ __forceinline__ void mma_lower(float (&d)[C / 8][4], const float (&s)[C / 8][4],
                                          uint32_t base, int lane) {
#pragma unroll
  for (int ks = 0; ks < C / 16; ++ks) {
    uint32_t f[NT][4];
    a_from<NT>(s[2 * ks], s[2 * ks + 1], f);
#pragma unroll
    for (int n = ks; n < C / 16; ++n)
      mma_apart<NT, NT, false>(d[2 * n], d[2 * n + 1], f, blockn_at<C>(base, n * 16, ks * 16, lane),
                              C * C * 2);
  }
}

// The warp's [16 channels, C tokens] through its piece of shared memory into rows
// of `ld` elements: value e of a token at dst + token * ld + e; tokens below
// rows, channels below cols.
template <typename T, int C>
__device__ __forceinline__ void store_rows(const float (&s)[C / 8][4], unsigned char* buf,
                                           uint32_t pitch, T* dst, int64_t ld, int rows, int cols,
                                           bool wide, int lane) {
  const int g = lane >> 2, t = lane & 3;
  __syncwarp();
#pragma unroll
  for (int n = 0; n < C / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<T*>(buf + (n * 8 + t * 2 + (e & 1)) * pitch +
                            (g + 8 * (e >> 1)) * sizeof(T)) = from_f<T>(s[n][e]);
  __syncwarp();
  constexpr int U = 16 * sizeof(T) / 16, E = 16 / sizeof(T);
  for (int i = lane; i < C * U; i += 32) {
    const int r = i / U, u = i % U;
    if (r >= rows) continue;
    const uint4 w = *reinterpret_cast<const uint4*>(buf + r * pitch + u * 16);
    T* p = dst + r * ld + u * E;
    if (wide && u * E + E <= cols) {
      *reinterpret_cast<uint4*>(p) = w;
    } else {
      const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (u * E + j < cols) p[j] = e[j];
    }
  }
}
// The same as bf16 terms into planes [C][VP] of the workspace.
template <int C, int NT>
__device__ __forceinline__ void store_terms(const float (&s)[C / 8][4], unsigned char* buf,
                                            uint32_t pitch, bf16* dst, int64_t ld, int64_t plane,
                                            int lane) {
  float r[C / 8][4];
#pragma unroll
  for (int n = 0; n < C / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) r[n][e] = s[n][e];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    float h[C / 8][4];   // the term
#pragma unroll
    for (int n = 0; n < C / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const uint32_t w = i + 1 < NT ? pack2_part(r[n][e], r[n][e + 1]) : pack2(r[n][e], r[n][e + 1]);
        h[n][e] = lo_of(w);
        h[n][e + 1] = hi_of(w);
        r[n][e] -= h[n][e];
        r[n][e + 1] -= h[n][e + 1];
      }
    store_rows<bf16, C>(h, buf, pitch, dst + i * plane, ld, C, 16, true, lane);
  }
}
// A warp's 16 rows of a state as terms into planes [VP][KP].
template <int KP, int NT>
__device__ __forceinline__ void store_state(const float (&s)[KP / 8][4], bf16* dst, int64_t plane,
                                            int lane) {
#pragma unroll
  for (int n = 0; n < KP / 8; ++n)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint32_t w[NT];
      split2<NT>(s[n][2 * r], s[n][2 * r + 1], w);
#pragma unroll
      for (int i = 0; i < NT; ++i)
        *reinterpret_cast<uint32_t*>(dst + i * plane + ((lane >> 2) + 8 * r) * KP + n * 8 +
                                     (lane & 3) * 2) = w[i];
    }
}
// ... and between registers and a dense [V, K] fp32 state.
template <int KP>
__device__ __forceinline__ void read_state(float (&s)[KP / 8][4], const float* src, int v0, int V,
                                           int K, int lane) {
#pragma unroll
  for (int n = 0; n < KP / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int v = v0 + (lane >> 2) + 8 * (e >> 1), k = n * 8 + (lane & 3) * 2 + (e & 1);
      s[n][e] = src && v < V && k < K ? src[(int64_t)v * K + k] : 0.f;
    }
}
template <int KP>
__device__ __forceinline__ void write_state(const float (&s)[KP / 8][4], float* dst, int v0, int V,
                                            int K, int lane) {
#pragma unroll
  for (int n = 0; n < KP / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int v = v0 + (lane >> 2) + 8 * (e >> 1), k = n * 8 + (lane & 3) * 2 + (e & 1);
      if (v < V && k < K) dst[(int64_t)v * K + k] = s[n][e];
    }
}

// How many have rows: all that a CTA can have share a chunk's tiles where the heads
// alone fill the SMs, fewer (and more CTAs) where they do not.
inline cudaError_t warps_for(const Args& a, int* warps) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int slices = a.VP / 16;
  int nw = slices < kRowWarps ? slices : kRowWarps;
  while (nw > 1 && (int64_t)a.B * a.H * ((slices + nw - 1) / nw) < sms) nw = (nw + 1) / 2;
  *warps = nw;
  return cudaSuccess;
}

}  // namespace delta
}  // namespace ssd
