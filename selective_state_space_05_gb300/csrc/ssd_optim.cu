// AdamW over many tensors at once (include/ssd_optim.h).
// Bound by HBM: each parameter's gradient, moments and value are read once, the
// moments and value written once.  As in ssd_clip.cu the tensors come as a table
// in the kernel's parameters (no copy to the device, capturable as is), cut into
// chunks that CTAs take a grid apart; a thread has eight elements of every tensor
// in flight.
//
// 643 M bf16 parameters with masters take 3.1 to 3.3 ms for 18 GB, 5.5 to 5.8 TB/s; four
// CTAs of 256 threads an SM were the fastest of 128 to 512 threads (3.2, 3.1, 3.1), and
// two groups of eight elements in flight a thread slower (3.4).
//
// 8-bit moments: a warp holds one block of 256 elements, eight a lane, so that the
// new scales are two reductions over the warp.  The arithmetic of m, v and their
// codes is in single rounded operations (no contraction), so that a code depends
// on nothing but its inputs.  Bound by instruction issue, a hundred an element: 161 M
// parameters take 0.85 ms (1.7 with divisions, exact roots and conversions), and their
// moments' values, which are HBM's, 0.28.
#include <math.h>
#include <stdio.h>

#include <algorithm>

#include "../../include/ssd_optim.h"
#include "ssd_common.cuh"
#include "ssd_row.cuh"

namespace ssd {
namespace optim {

using bf16 = __nv_bfloat16;
constexpr int kThreads = 256, kVec = row::kVec;
constexpr int kChunk = 8192;                // elements
constexpr int kBlock = SSD_ADAMW_BLOCK;
static_assert(kBlock == 32 * kVec, "a warp holds a block");
constexpr int kSmall = 40, kLarge = 360;    // tensors a launch: 3 KB or 28 KB of parameters
template <int BITS>
constexpr int kCtas = BITS == 8 ? 3 : 4;    // an SM

enum { kParamBf16 = 1, kGradBf16 = 2, kMaster = 4 };
struct Entry {
  void* p;
  const void* g;
  float* master;
  void *m, *v;
  float *ms, *vs;
  int64_t n;
  uint32_t first, num;   // first chunk in this launch; number in the list
  uint32_t flags, pad;
};
template <int N>
struct Table {
  Entry e[N];
  uint32_t tensors, chunks;
};

struct Opt {
  double lr, log_b1, log_b2, decay, step;
  const int64_t* step_dev;
  const float *lr_dev, *norm;
  float b1, c1, b2, c2, eps, max_norm;   // c = 1 - b
  uint32_t seed, step_low;
};
// What each thread needs of it.
struct Factors {
  float size, keep, root;   // lr / (1 - beta1^t), 1 - lr decay, (1 - beta2^t)^-1/2
  // clipping: coef * first, where first is 1, or 2^-64 where the factor alone would be a
  // subnormal of few bits (ssd_clip.cu)
  float coef, first;
  uint32_t key;
};

__device__ __forceinline__ uint32_t mix(uint32_t h) {
  h = (h ^ (h >> 16)) * 0x7FEB352Du;
  h = (h ^ (h >> 15)) * 0x846CA68Bu;
  return h ^ (h >> 16);
}

// By one thread of a CTA.
__device__ __forceinline__ Factors factors(const Opt& o) {
  Factors f;
  double t = o.step, lr = o.lr;
  uint32_t low = o.step_low;
  if (o.step_dev) {
    const int64_t s = *o.step_dev;
    t = (double)s;
    low = (uint32_t)s;
  }
  if (o.lr_dev) lr = (double)*o.lr_dev;
  f.size = (float)(lr / -expm1(t * o.log_b1));
  f.root = (float)(1.0 / sqrt(-expm1(t * o.log_b2)));
  f.keep = (float)(1.0 - lr * o.decay);
  f.coef = f.first = 1.f;
  if (o.norm) {
    // (a product with the reciprocal: what a tensor under a number is elsewhere)
    const float r = __frcp_rn(__fadd_rn(*o.norm, 1e-6f));
    float c = __fmul_rn(r, o.max_norm);
    if (r < 0x1p-126f || c < 0x1p-100f) {   // near the end of the range: as clip_grads
      const double d = (double)o.max_norm / ((double)*o.norm + 1e-6);
      const bool tiny = d < 0x1p-100;
      f.first = tiny ? 0x1p-64f : 1.f;
      c = (float)(tiny ? d * 0x1p64 : d);
    }
    f.coef = c >= 1.f ? 1.f : c;   // a NaN norm gives NaN
  }
  f.key = mix(mix(o.seed) + low);
  return f;
}

template <int N>
__device__ __forceinline__ uint32_t tensor_of(const Table<N>& t, uint32_t chunk) {
  uint32_t lo = 0, hi = t.tensors;   // the last tensor whose first chunk is <= chunk
  while (hi - lo > 1) {
    const uint32_t m = (lo + hi) / 2;
    if (t.e[m].first <= chunk) lo = m;
    else hi = m;
  }
  return lo;
}

__device__ __forceinline__ void load8(const float* p, bool wide, float (&v)[kVec]) {
  if (wide) {
    row::load_slot<true>(p, 0, 0, 1, kVec, v);
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = p[j];
  }
}
__device__ __forceinline__ void load8(const bf16* p, bool wide, float (&v)[kVec]) {
  if (wide) {
    row::load_slot<true>(p, 0, 0, 1, kVec, v);
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = __bfloat162float(p[j]);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, bool wide, const float (&v)[kVec]) {
  if (wide) {
    row::store_slot<true>(p, 0, 0, 1, kVec, v);
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) p[j] = from_f<T>(v[j]);
  }
}
__device__ __forceinline__ bool on16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Gradients as clipping leaves them.
__device__ __forceinline__ void clip(float (&g)[kVec], const Factors& f) {
  if (f.first != 1.f) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) g[j] = __fmul_rn(g[j], f.first);
  }
#pragma unroll
  for (int j = 0; j < kVec; ++j) g[j] = __fmul_rn(g[j], f.coef);
}
__device__ __forceinline__ void moments(float g, float& m, float& v, const Opt& o) {
  m = __fadd_rn(__fmul_rn(m, o.b1), __fmul_rn(g, o.c1));
  v = __fadd_rn(__fmul_rn(v, o.b2), __fmul_rn(__fmul_rn(g, g), o.c2));
}
__device__ __forceinline__ float root(float v) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// (the root and the division are within 2^-21, which is nothing beside p's own
// rounding: a step moves p by lr)
__device__ __forceinline__ float update(float p, float m, float v, const Factors& f,
                                        const Opt& o) {
  return fmaf(p, f.keep, -__fdividef(m * f.size, fmaf(root(v), f.root, o.eps)));
}

// Elements [at, at + n) of a tensor, moments in fp32.
template <typename P, typename G, bool MASTER>
__device__ __forceinline__ void chunk32(const Entry& e, int64_t at, int n, const Factors& f,
                                        const Opt& o) {
  P* const p = static_cast<P*>(e.p) + at;
  const G* const g = static_cast<const G*>(e.g) + at;
  float* const w = MASTER ? e.master + at : nullptr;
  float* const m = static_cast<float*>(e.m) + at;
  float* const v = static_cast<float*>(e.v) + at;
  // eight-element groups begin where m's 32 bytes do; the others' places there
  // are wide too when the tensors were cut from buffers alike
  const int skip = (int)(((32 - ((uintptr_t)m & 31)) & 31) / 4), head = skip < n ? skip : n;
  const bool wg = on16(g + head), wp = on16(p + head), wv = on16(v + head),
             ww = MASTER && on16(w + head);
  const int vecs = (n - head) / kVec;
  for (int i = threadIdx.x; i < vecs; i += kThreads) {
    const int k = head + i * kVec;
    float gv[kVec], mv[kVec], vv[kVec], pv[kVec];
    load8(g + k, wg, gv);
    load8(m + k, true, mv);
    load8(v + k, wv, vv);
    if (MASTER) load8(w + k, ww, pv);
    else load8(p + k, wp, pv);
    clip(gv, f);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      moments(gv[j], mv[j], vv[j], o);
      pv[j] = update(pv[j], mv[j], vv[j], f, o);
    }
    store8(m + k, true, mv);
    store8(v + k, wv, vv);
    if (MASTER) store8(w + k, ww, pv);
    store8(p + k, wp, pv);
  }
  // the ends, one element a thread
  const int tail = n - head - vecs * kVec;
  if ((int)threadIdx.x < head + tail) {
    const int k = (int)threadIdx.x < head ? threadIdx.x : threadIdx.x + vecs * kVec;
    float mv = m[k], vv = v[k];
    moments(__fmul_rn(__fmul_rn(to_f(g[k]), f.first), f.coef), mv, vv, o);
    const float pv = update(MASTER ? w[k] : to_f(p[k]), mv, vv, f, o);
    m[k] = mv;
    v[k] = vv;
    if (MASTER) w[k] = pv;
    p[k] = from_f<P>(pv);
  }
}

// ------------------------------------------------------------------ 8 bits
// Small whole numbers and floats, through the bits of 2^23 + n (conversion
// instructions run at a quarter of the rate).
__device__ __forceinline__ float float_of(uint32_t word, int byte) {
  return __uint_as_float(__byte_perm(word, 0x4B000000u, 0x7440u + byte)) - 8388608.f;
}
// A word of four whole n in [0, 256], 256 as 0.
__device__ __forceinline__ uint32_t word_of(float a, float b, float c, float d) {
  auto bits = [](float x) { return __float_as_uint(x + 8388608.f); };
  return __byte_perm(__byte_perm(bits(a), bits(b), 0x0040), __byte_perm(bits(c), bits(d), 0x0040),
                     0x5410);
}
__device__ __forceinline__ float floor_of(float x) {   // of 0 <= x < 2^22
  return __fadd_rz(x, 8388608.f) - 8388608.f;
}
__device__ __forceinline__ float share(uint32_t n) {   // (n + 1/2) 2^-16, n < 2^16
  return (__uint_as_float(0x4B000000u | n) - 8388607.5f) * 0x1p-16f;
}
__device__ __forceinline__ float m_unit(float c) {   // of a code's size
  const float t = __fmul_rn(c, 1.0f / 127.0f);
  return __fmul_rn(t, t);
}
__device__ __forceinline__ float v_unit(float c) {
  const float t = __fmul_rn(c, 1.0f / 255.0f), s = __fmul_rn(t, t);
  return __fmul_rn(s, s);
}
// A signed code's value; `word` has 128 added to each.
__device__ __forceinline__ float m_of(uint32_t word, int byte) {
  const float t = __fmul_rn(float_of(word, byte) - 128.f, 1.0f / 127.0f);
  return __fmul_rn(t, fabsf(t));
}
// The code of x >= 0 below the largest: the one below it, or the next with the odds
// that keep its value, u in (0, 1); x's quotient by the largest, the place of its
// root among the codes and the odds are each rounded to nearest.
template <bool SQUARE>
__device__ __forceinline__ float code_of(float x, float big, float u) {
  constexpr float top = SQUARE ? 127.f : 255.f;
  const float r = x > 0.f ? __fdiv_rn(x, big) : 0.f;
  const float y = SQUARE ? __fsqrt_rn(r) : __fsqrt_rn(__fsqrt_rn(r));
  const float c = fminf(floorf(__fmul_rn(y, top)), top - 1.f);
  const float lo = SQUARE ? m_unit(c) : v_unit(c), hi = SQUARE ? m_unit(c + 1.f) : v_unit(c + 1.f);
  return u < __fdiv_rn(__fsub_rn(r, lo), __fsub_rn(hi, lo)) ? c + 1.f : c;
}
// The same without its divisions and roots, u = (2 n + 1) 2^-17 with n < 2^16.  The
// quotient is Markstein's correction of the product with the largest's rounded
// reciprocal (largest and quotient well within the normal range).  The odds round to
// more than u where they are above it by more than half of u's last place, which the
// sign of n - u d tells.  The approximate root, within 2^-13 of its place among the
// codes, is on the wrong side of one only where x is next to that code's value; then
// both sides give the same code but for u next to 0 or 1: `unsure` is above 0.499
// there (four in a million), and code_of is asked.
__device__ __forceinline__ float quick_root(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
template <bool SQUARE>
__device__ __forceinline__ float quick_code(float x, float big, float inv, float u, float& unsure) {
  constexpr float top = SQUARE ? 127.f : 255.f;
  const float q = x * inv, r = fmaf(fmaf(-q, big, x), inv, q);
  const float y = fminf((SQUARE ? quick_root(r) : quick_root(quick_root(r))) * top, top);
  const float c = fminf(floor_of(y), top - 1.f);
  unsure = fmaxf(unsure, fminf(fabsf(y - c - 0.5f), fabsf(u - 0.5f)));
  const float lo = SQUARE ? m_unit(c) : v_unit(c), hi = SQUARE ? m_unit(c + 1.f) : v_unit(c + 1.f);
  const float step = __fsub_rn(hi, lo);
  const float half = __uint_as_float((__float_as_uint(u) & 0x7F800000u) - (24u << 23));
  return fmaf(-half, step, fmaf(-u, step, __fsub_rn(r, lo))) > 0.f ? c + 1.f : c;
}
// The largest of 256 magnitudes (a NaN is larger than all).
__device__ __forceinline__ float warp_max(const float (&x)[kVec]) {
  uint32_t b = 0;
#pragma unroll
  for (int j = 0; j < kVec; ++j) b = max(b, __float_as_uint(x[j]) & 0x7FFFFFFFu);
  return __uint_as_float(__reduce_max_sync(0xffffffffu, b));
}

__device__ __forceinline__ void load_codes(const uint8_t* p, bool wide, int n, uint2& w) {
  if (wide) {
    w = *reinterpret_cast<const uint2*>(p);
  } else {
    w = make_uint2(0, 0);
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (j < n) (j < 4 ? w.x : w.y) |= (uint32_t)p[j] << (j % 4 * 8);
  }
}
__device__ __forceinline__ void store_codes(uint8_t* p, bool wide, int n, uint2 w) {
  if (wide) {
    *reinterpret_cast<uint2*>(p) = w;
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (j < n) p[j] = (uint8_t)((j < 4 ? w.x : w.y) >> (j % 4 * 8));
  }
}
__device__ __forceinline__ bool on8(const void* p) { return ((uintptr_t)p & 7) == 0; }

// n of eight values (all of them: wide where on 16 bytes).
template <typename T>
__device__ __forceinline__ void load_some(const T* p, int n, float (&v)[kVec]) {
  if (n == kVec) {
    load8(p, on16(p), v);
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = j < n ? to_f(p[j]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store_some(T* p, int n, const float (&v)[kVec]) {
  if (n == kVec) {
    store8(p, on16(p), v);
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (j < n) p[j] = from_f<T>(v[j]);
  }
}

template <typename P, typename G, bool MASTER>
__device__ __forceinline__ void chunk8(const Entry& e, int64_t at, int n, const Factors& f,
                                       const Opt& o) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int k0 = warp * kBlock; k0 < n; k0 += kThreads / 32 * kBlock) {
    const int64_t i = at + k0 + lane * kVec;    // the lane's first element
    const int64_t blk = (at + k0) / kBlock;
    const int left = (int)(e.n - i < kVec ? (e.n > i ? e.n - i : 0) : kVec);
    P* const p = static_cast<P*>(e.p) + i;
    float* const w = MASTER ? e.master + i : nullptr;
    uint8_t* const mc = static_cast<uint8_t*>(e.m) + i;
    uint8_t* const vc = static_cast<uint8_t*>(e.v) + i;
    const float ms = e.ms[blk], vs = e.vs[blk];
    float gv[kVec], pv[kVec], mv[kVec], vv[kVec];
    uint2 cm, cv;
    const bool full = left == kVec;
    load_some(static_cast<const G*>(e.g) + i, left, gv);
    load_codes(mc, full && on8(mc), left, cm);
    load_codes(vc, full && on8(vc), left, cv);
    cm.x ^= 0x80808080u;
    cm.y ^= 0x80808080u;
    if (MASTER) load_some(w, left, pv);
    else load_some(p, left, pv);
    clip(gv, f);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      mv[j] = __fmul_rn(m_of(j < 4 ? cm.x : cm.y, j % 4), ms);
      vv[j] = __fmul_rn(v_unit(float_of(j < 4 ? cv.x : cv.y, j % 4)), vs);
      if (j >= left) mv[j] = vv[j] = 0.f;   // (a scale that is not finite stays out of the rest)
      moments(gv[j], mv[j], vv[j], o);
      if (j >= left) mv[j] = vv[j] = 0.f;
      pv[j] = update(pv[j], mv[j], vv[j], f, o);
    }
    if (MASTER) store_some(w, left, pv);
    store_some(p, left, pv);
    const float mb = warp_max(mv), vb = warp_max(vv);
    const float mi = mb > 0.f ? __frcp_rn(mb) : 0.f, vi = vb > 0.f ? __frcp_rn(vb) : 0.f;
    auto usual = [](float x) { return x == 0.f || (x > 0x1p-90f && x < 0x1p90f); };
    const bool plain = usual(mb) && usual(vb);
    float unsure = plain ? 0.f : 1.f;
    uint32_t key = mix(f.key + e.num);
    if (i >> 32) key = mix(key + (uint32_t)(i >> 32));
    float a[kVec], b[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const uint32_t h = mix(key + (uint32_t)i + j);
      a[j] = quick_code<true>(fabsf(mv[j]), mb, mi, share(h >> 16), unsure);
      b[j] = quick_code<false>(vv[j], vb, vi, share(h & 0xFFFFu), unsure);
    }
    if (unsure > 0.499f) {
#pragma unroll 1
      for (int k = 0; k < kVec; ++k) {   // (a loop, and picks, for few registers)
        float x = mv[0], z = vv[0];
#pragma unroll
        for (int j = 1; j < kVec; ++j) {
          x = j == k ? mv[j] : x;
          z = j == k ? vv[j] : z;
        }
        const uint32_t h = mix(key + (uint32_t)i + k);
        x = code_of<true>(fabsf(x), mb, share(h >> 16));
        z = code_of<false>(z, vb, share(h & 0xFFFFu));
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          a[j] = j == k ? x : a[j];
          b[j] = j == k ? z : b[j];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      a[j] = mv[j] < 0.f ? 256.f - a[j] : a[j];
      b[j] = vv[j] > 0.f ? fmaxf(b[j], 1.f) : b[j];
    }
    cm = make_uint2(word_of(a[0], a[1], a[2], a[3]), word_of(a[4], a[5], a[6], a[7]));
    cv = make_uint2(word_of(b[0], b[1], b[2], b[3]), word_of(b[4], b[5], b[6], b[7]));
    store_codes(mc, full && on8(mc), left, cm);
    store_codes(vc, full && on8(vc), left, cv);
    if (lane == 0) {
      e.ms[blk] = mb;
      e.vs[blk] = vb;
    }
  }
}

template <int BITS, typename P, typename G, bool MASTER>
__device__ __forceinline__ void chunk(const Entry& e, int64_t at, int n, const Factors& f,
                                      const Opt& o) {
  if constexpr (BITS == 32) chunk32<P, G, MASTER>(e, at, n, f, o);
  else chunk8<P, G, MASTER>(e, at, n, f, o);
}

template <int N, int BITS>
__global__ void __launch_bounds__(kThreads, kCtas<BITS>)
    step_kernel(const __grid_constant__ Table<N> t, const __grid_constant__ Opt o) {
  __shared__ Factors sf;
  if (threadIdx.x == 0) sf = factors(o);
  __syncthreads();
  const Factors f = sf;
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const Entry& e = t.e[tensor_of(t, c)];
    const int64_t at = (int64_t)(c - e.first) * kChunk, left = e.n - at;
    const int n = (int)(left < kChunk ? left : kChunk);
    const uint32_t k = e.flags;
    if (k & kMaster) {
      if (k & kParamBf16) {
        if (k & kGradBf16) chunk<BITS, bf16, bf16, true>(e, at, n, f, o);
        else chunk<BITS, bf16, float, true>(e, at, n, f, o);
      } else {
        if (k & kGradBf16) chunk<BITS, float, bf16, true>(e, at, n, f, o);
        else chunk<BITS, float, float, true>(e, at, n, f, o);
      }
    } else if (k & kParamBf16) {
      if (k & kGradBf16) chunk<BITS, bf16, bf16, false>(e, at, n, f, o);
      else chunk<BITS, bf16, float, false>(e, at, n, f, o);
    } else {
      if (k & kGradBf16) chunk<BITS, float, bf16, false>(e, at, n, f, o);
      else chunk<BITS, float, float, false>(e, at, n, f, o);
    }
  }
}

// 8-bit moments' values; the table's p and master are where they go.
template <int N>
__global__ void __launch_bounds__(kThreads) values_kernel(const __grid_constant__ Table<N> t) {
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const Entry& e = t.e[tensor_of(t, c)];
    const int64_t at = (int64_t)(c - e.first) * kChunk, end = std::min(e.n, at + kChunk);
    for (int64_t i = at + threadIdx.x * kVec; i < end; i += kThreads * kVec) {
      const int left = (int)(end - i < kVec ? end - i : kVec);
      const uint8_t *mc = static_cast<const uint8_t*>(e.m) + i,
                    *vc = static_cast<const uint8_t*>(e.v) + i;
      const float ms = e.ms[i / kBlock], vs = e.vs[i / kBlock];
      uint2 cm, cv;
      load_codes(mc, left == kVec && on8(mc), left, cm);
      load_codes(vc, left == kVec && on8(vc), left, cv);
      cm.x ^= 0x80808080u;
      cm.y ^= 0x80808080u;
      float mv[kVec], vv[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        mv[j] = __fmul_rn(m_of(j < 4 ? cm.x : cm.y, j % 4), ms);
        vv[j] = __fmul_rn(v_unit(float_of(j < 4 ? cv.x : cv.y, j % 4)), vs);
      }
      store_some(static_cast<float*>(e.p) + i, left, mv);
      store_some(e.master + i, left, vv);
    }
  }
}

int bad(int code, const char* msg) { return set_error(code, msg); }
bool off(const void* p, size_t align) { return ((uintptr_t)p & (align - 1)) != 0; }

// Fills the next launch's table from tensor `k` on; returns the tensor after it.
template <int N, typename F>
int fill(Table<N>& t, int k, int count, const int64_t* n, F entry) {
  t.tensors = t.chunks = 0;
  for (; k < count && t.tensors < N; ++k) {
    if (n[k] == 0) continue;
    const int64_t chunks = (n[k] + kChunk - 1) / kChunk;
    if (t.tensors > 0 && t.chunks + chunks > 0x7fffffff) break;
    Entry& e = t.e[t.tensors++];
    e = entry(k);
    e.n = n[k];
    e.first = t.chunks;
    e.num = (uint32_t)k;
    t.chunks += (uint32_t)chunks;
  }
  return k;
}
int grid_of(uint32_t chunks, int ctas) {
  return (int)std::min<int64_t>(chunks, (int64_t)row::sm_count() * ctas);
}
int launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return SSD_OK;
  char m[256];
  snprintf(m, sizeof(m), "%s launch: %s", what, cudaGetErrorString(e));
  return set_error(SSD_ERR_CUDA, m);
}

template <int N, typename F>
int run_step(const int64_t* n, int count, int bits, const Opt& o, F entry, cudaStream_t st) {
  static thread_local Table<N> t;   // too large for some callers' stacks
  for (int k = 0; k < count;) {
    k = fill(t, k, count, n, entry);
    if (t.chunks == 0) break;
    if (bits == 32) step_kernel<N, 32><<<grid_of(t.chunks, kCtas<32>), kThreads, 0, st>>>(t, o);
    else step_kernel<N, 8><<<grid_of(t.chunks, kCtas<8>), kThreads, 0, st>>>(t, o);
  }
  return launched("adamw_step");
}
template <int N, typename F>
int run_values(const int64_t* n, int count, F entry, cudaStream_t st) {
  static thread_local Table<N> t;
  for (int k = 0; k < count;) {
    k = fill(t, k, count, n, entry);
    if (t.chunks == 0) break;
    values_kernel<N><<<grid_of(t.chunks, kCtas<32>), kThreads, 0, st>>>(t);
  }
  return launched("adamw_moments");
}

}  // namespace optim
}  // namespace ssd

using namespace ssd::optim;

extern "C" {

int ssd_optim_abi_version(void) { return SSD_OPTIM_ABI_VERSION; }

int ssd_adamw_step(void* const* params, const int32_t* param_dtypes, const void* const* grads,
                   const int32_t* grad_dtypes, float* const* masters, void* const* exp_avgs,
                   void* const* exp_avg_sqs, float* const* exp_avg_scales,
                   float* const* exp_avg_sq_scales, const int64_t* sizes, int count, int bits,
                   const ssd_adamw_t* options, void* stream) {
  if (count < 0) return bad(SSD_ERR_ARG, "count must be >= 0");
  if (bits != 32 && bits != 8) return bad(SSD_ERR_ARG, "bits must be 32 or 8");
  if (!options) return bad(SSD_ERR_NULL, "options are required");
  const ssd_adamw_t& u = *options;
  if (!(u.beta1 >= 0.0 && u.beta1 < 1.0) || !(u.beta2 >= 0.0 && u.beta2 < 1.0))
    return bad(SSD_ERR_ARG, "betas must be in [0, 1)");
  if (!(u.eps >= 0.0) || !(u.weight_decay >= 0.0) || !(fabs(u.lr) < INFINITY) ||
      u.eps > 3e38 || u.weight_decay > 3e38)
    return bad(SSD_ERR_ARG, "eps and weight_decay must be >= 0, lr finite");
  if (!u.step_dev && u.step < 1) return bad(SSD_ERR_ARG, "step must be >= 1");
  if (u.grad_norm && !(u.max_norm >= 0.0)) return bad(SSD_ERR_ARG, "max_norm must be >= 0");
  if (off(u.step_dev, 8) || off(u.lr_dev, 4) || off(u.grad_norm, 4))
    return bad(SSD_ERR_ALIGN, "a pointer is not aligned to its element");
  if (count > 0 && (!params || !param_dtypes || !grads || !grad_dtypes || !exp_avgs ||
                    !exp_avg_sqs || !sizes || (bits == 8 && (!exp_avg_scales || !exp_avg_sq_scales))))
    return bad(SSD_ERR_NULL, "an array is NULL");
  for (int k = 0; k < count; ++k) {
    if (sizes[k] < 0) return bad(SSD_ERR_ARG, "sizes must be >= 0");
    if (sizes[k] > (1LL << 43)) return bad(SSD_ERR_UNSUPPORTED, "a size is above 2^43");
    if (sizes[k] == 0) continue;
    const int32_t pt = param_dtypes[k], gt = grad_dtypes[k];
    if ((pt != SSD_DTYPE_F32 && pt != SSD_DTYPE_BF16) || (gt != SSD_DTYPE_F32 && gt != SSD_DTYPE_BF16))
      return bad(SSD_ERR_ARG, "unknown dtype");
    if (!params[k] || !grads[k] || !exp_avgs[k] || !exp_avg_sqs[k] ||
        (bits == 8 && (!exp_avg_scales[k] || !exp_avg_sq_scales[k])))
      return bad(SSD_ERR_NULL, "a parameter, gradient, moment or scale is NULL");
    const size_t me = bits == 32 ? 4 : 1;
    if (off(params[k], pt == SSD_DTYPE_BF16 ? 2 : 4) || off(grads[k], gt == SSD_DTYPE_BF16 ? 2 : 4) ||
        off(exp_avgs[k], me) || off(exp_avg_sqs[k], me) || (masters && off(masters[k], 4)) ||
        (bits == 8 && (off(exp_avg_scales[k], 4) || off(exp_avg_sq_scales[k], 4))))
      return bad(SSD_ERR_ALIGN, "a pointer is not aligned to its element");
  }
  Opt o = {};
  o.lr = u.lr;
  o.log_b1 = log(u.beta1);
  o.log_b2 = log(u.beta2);
  o.decay = u.weight_decay;
  o.step = (double)u.step;
  o.step_dev = u.step_dev;
  o.lr_dev = u.lr_dev;
  o.norm = u.grad_norm;
  o.b1 = (float)u.beta1;
  o.c1 = (float)(1.0 - u.beta1);
  o.b2 = (float)u.beta2;
  o.c2 = (float)(1.0 - u.beta2);
  o.eps = (float)u.eps;
  o.max_norm = (float)u.max_norm;
  o.seed = u.seed;
  o.step_low = (uint32_t)u.step;
  auto entry = [&](int k) {
    Entry e = {};
    e.p = params[k];
    e.g = grads[k];
    e.master = masters ? masters[k] : nullptr;
    e.m = exp_avgs[k];
    e.v = exp_avg_sqs[k];
    if (bits == 8) {
      e.ms = exp_avg_scales[k];
      e.vs = exp_avg_sq_scales[k];
    }
    e.flags = (param_dtypes[k] == SSD_DTYPE_BF16 ? kParamBf16 : 0) |
              (grad_dtypes[k] == SSD_DTYPE_BF16 ? kGradBf16 : 0) | (e.master ? kMaster : 0);
    return e;
  };
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return count <= kSmall ? run_step<kSmall>(sizes, count, bits, o, entry, st)
                         : run_step<kLarge>(sizes, count, bits, o, entry, st);
}

int ssd_adamw_moments(const void* const* exp_avgs, const void* const* exp_avg_sqs,
                      const float* const* exp_avg_scales, const float* const* exp_avg_sq_scales,
                      float* const* exp_avg_values, float* const* exp_avg_sq_values,
                      const int64_t* sizes, int count, void* stream) {
  if (count < 0) return bad(SSD_ERR_ARG, "count must be >= 0");
  if (count > 0 && (!exp_avgs || !exp_avg_sqs || !exp_avg_scales || !exp_avg_sq_scales ||
                    !exp_avg_values || !exp_avg_sq_values || !sizes))
    return bad(SSD_ERR_NULL, "an array is NULL");
  for (int k = 0; k < count; ++k) {
    if (sizes[k] < 0) return bad(SSD_ERR_ARG, "sizes must be >= 0");
    if (sizes[k] > (1LL << 43)) return bad(SSD_ERR_UNSUPPORTED, "a size is above 2^43");
    if (sizes[k] == 0) continue;
    if (!exp_avgs[k] || !exp_avg_sqs[k] || !exp_avg_scales[k] || !exp_avg_sq_scales[k] ||
        !exp_avg_values[k] || !exp_avg_sq_values[k])
      return bad(SSD_ERR_NULL, "a moment, scale or output is NULL");
    if (off(exp_avg_scales[k], 4) || off(exp_avg_sq_scales[k], 4) || off(exp_avg_values[k], 4) ||
        off(exp_avg_sq_values[k], 4))
      return bad(SSD_ERR_ALIGN, "a pointer is not aligned to its element");
  }
  auto entry = [&](int k) {
    Entry e = {};
    e.p = exp_avg_values[k];
    e.master = exp_avg_sq_values[k];
    e.m = const_cast<void*>(exp_avgs[k]);
    e.v = const_cast<void*>(exp_avg_sqs[k]);
    e.ms = const_cast<float*>(exp_avg_scales[k]);
    e.vs = const_cast<float*>(exp_avg_sq_scales[k]);
    return e;
  };
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return count <= kSmall ? run_values<kSmall>(sizes, count, entry, st)
                         : run_values<kLarge>(sizes, count, entry, st);
}

}  // extern "C"
