// What the gated delta rule's kernels share: their sizes and workspace, bf16
// tiles in shared memory, and products of values kept as sums of bf16 terms.
//
// Per batch row and head, with S [headdim, dstate], tokens in chunks of C:
//   S' = e^g S,  u = beta (v - S' k),  S = S' + u k^T,  out = scale S q
// With G the sum of g from the chunk's start and D_ij = e^(G_i - G_j), i >= j:
//   N = strict lower D k k^T,  T = (I + N diag(beta))^-1,  P = scale lower D q k^T
//   x = T (v - e^G S0 k),  u = beta x,  out = scale e^G S0 q + P u
//   S_C = e^(G_C) S0 + sum_j e^(G_C - G_j) u_j k_j^T
//
// Products have bf16 operands and fp32 sums.  Inputs in bf16 are one term; what is
// computed in fp32 (the state, x, u, T, P and their gradients) is split into NT bf16
// terms, each the rounding of what the ones before leave, and the products a_i b_j
// with i + j < NT are summed: two terms leave 2^-18 of each factor, which is nothing
// beside what bf16 inputs and outputs round; three (for fp32 inputs, themselves three
// terms) about 2^-26.
//
// bf16 runs on tcgen05 (ssd_delta_tc*): for 8 x 1024 tokens of 128 heads of 32
// channels and a dstate of 32 the forward takes 0.59 ms there and 0.95 with mma.sync,
// forward and backward 1.82 and 2.74, and no size was found where it is the slower one by
// more than a microsecond.  fp32 runs on mma.sync m16n8k16: six products a pair of
// factors, whose three terms would not fit TMEM beside the results; a warp owns 16 of
// the state's rows, and its accumulators are, register by register, the A operand of
// the next mma, so that a chunk's chain of five products meets no memory and no other
// warp.  (mma.sync runs bf16 at 593 TFLOP/s on all SMs, one m16n8k16 per 8 cycles and
// quadrant.)
#pragma once

#include "ssd_common.cuh"

namespace ssd {
namespace delta {

using bf16 = __nv_bfloat16;

// Chunk length and terms: bf16 inputs 64 tokens, two terms; fp32 32 and three
// (their tiles take three times the shared memory).
template <typename T> struct Mode;
template <> struct Mode<bf16> { static constexpr int C = 64, NT = 2; };
template <> struct Mode<float> { static constexpr int C = 32, NT = 3, TI = 3; };

// e^g is 0 in fp32 below this: such a token starts the state anew, as one
// whose seq_idx changes.
constexpr float kReset = -104.f;

// How the tcgen05 passes take a sequence's segments: one after another, each from the
// state that the one before left; or all at once, which takes two passes.  The first
// gives each segment's effect on a state, S -> S M + W: W from a state of zeros, M
// from the unit rows and without values.  Those are joined, and the second pass
// starts each segment from its own state.  (Backward: segments from the sequence's end,
// the state's gradient in S's place and dout in the values'.)
enum { kWhole, kParts, kJoined };

// Per chunk and head: vectors of C floats each, then e^(G_C) alone.
// e^G, e^(G_C - G), beta, G in two floats, the resets before a token; beta e^(G_C - G)
// and -e^G
enum { kGam, kOnto, kBeta, kGhi, kGlo, kSeg, kWrite, kRead, kVecs };
template <int C> constexpr int vec_floats() { return kVecs * C + 4; }

struct Args {
  int64_t L;
  int B, H, G, K, V, nc, KP, VP;   // KP: dstate padded to 64 or 128; VP: headdim to 16 or 128
  TokStride sq, sk, sv, sdo;
  int qcols, kcols, vcols, docols;   // dstate and headdim as their rows have them (packed: to 8)
  int wide_q, wide_k, wide_v, wide_do, wide_out, wide_dv;   // rows in 16-byte pieces
  int tc;       // bf16: the tcgen05 kernels and their workspace's layout
  float scale;
  const void *q, *k, *v, *dout;
  const float *g, *beta;
  const int32_t* seq;
  const float *init, *dfinal;
  void *out, *dv;
  float *final, *dinit;
  // workspace, per (batch row, head, chunk)
  bf16 *T, *P;     // [NT][C][C]
  float* vec;      // vec_floats
  bf16 *S0, *X;    // [NT][VP][KP], [NT][C][VP]; null in a forward that keeps nothing
  bf16 *dS, *dY;   // the same of the backward
  // the tcgen05 kernels' work: sequences in `segs` segments of `seg` chunks, a ticket
  // and one flag for each (head, 128 channels), and its state between segments
  int segs, seg;
  int pass;        // kWhole; or of a few long sequences, kParts and then kJoined
  int* ctrl;
  float *slots, *first;   // first: a copy of the first state (kParts)
  // gradients; per head [B, L, H, dstate] fp32 where heads share queries and keys
  void *dq, *dk;
  float *dg, *dbeta, *dq_part, *dk_part;
};

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t saddr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ------------------------------------------------------------------ tiles
// A tile of rows of W bf16 (W 16, 32, 64 or 128), 16-byte units swizzled so that
// eight rows' units of one column lie in eight bank groups.
template <int W>
__device__ __forceinline__ uint32_t tile_at(int row, int unit) {
  constexpr int U = W / 8;
  const int x = U >= 8 ? (row & 7) : U == 4 ? ((row >> 1) & 3) : ((row >> 2) & 1);
  return (uint32_t)(row * U + (unit ^ x)) * 16u;
}
// ldmatrix address of the 16 x 16 block at (row, col): lanes 0-7 rows 0-7 of the
// left unit, 8-15 rows 8-15 of it, then the right unit's.  Read plainly as an A
// operand [m][k]: a0..a3.  With .trans as a B operand stored [k][n]: {b0, b1} of
// the left 8 columns in r0, r1, of the right ones in r2, r3; as an A operand
// stored [k][m] see a_from_t.
template <int W>
__device__ __forceinline__ uint32_t block_at(uint32_t base, int row, int col, int lane) {
  return base + tile_at<W>(row + (lane & 15), (col >> 3) + (lane >> 4));
}
// The same block read plainly as a B operand stored [n][k]: {b0, b1} of rows
// 0-7 in r0, r1 and of rows 8-15 in r2, r3.
template <int W>
__device__ __forceinline__ uint32_t blockn_at(uint32_t base, int row, int col, int lane) {
  return base + tile_at<W>(row + (lane & 7) + ((lane >> 4) << 3), (col >> 3) + ((lane >> 3) & 1));
}

// ------------------------------------------------------------------ terms
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The same for a term that others follow: what is beyond bf16's largest value (finite
// ones within half a place of 2^128, and infinities) becomes that, and the rest is left
// to the next term, so that a finite value's terms are finite.
__device__ __forceinline__ uint32_t pack2_part(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// Two values as NT packed pairs of terms.
template <int NT>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&t)[NT]) {
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    t[i] = i + 1 < NT ? pack2_part(x, y) : pack2(x, y);
    if (i + 1 < NT) {
      x -= lo_of(t[i]);
      y -= hi_of(t[i]);
    }
  }
}
// A operand of 16 columns from two accumulator tiles (the left and right 8).
template <int NT>
__device__ __forceinline__ void a_from(const float (&l)[4], const float (&r)[4],
                                       uint32_t (&a)[NT][4]) {
  uint32_t t[NT];
  split2<NT>(l[0], l[1], t);
#pragma unroll
  for (int i = 0; i < NT; ++i) a[i][0] = t[i];
  split2<NT>(l[2], l[3], t);
#pragma unroll
  for (int i = 0; i < NT; ++i) a[i][1] = t[i];
  split2<NT>(r[0], r[1], t);
#pragma unroll
  for (int i = 0; i < NT; ++i) a[i][2] = t[i];
  split2<NT>(r[2], r[3], t);
#pragma unroll
  for (int i = 0; i < NT; ++i) a[i][3] = t[i];
}
// d0 += a b for two neighbouring n tiles, over the terms' products (indexes' sum
// below the larger number), smallest first.  B: planes of a tile in shared memory,
// `plane` bytes apart, at the address of its first plane; TR: stored [k][n].
template <int NA, int NB, bool TR>
__device__ __forceinline__ void mma_pair(float (&d0)[4], float (&d1)[4],
                                         const uint32_t (&a)[NA][4], uint32_t addr,
                                         uint32_t plane) {
  constexpr int N = NA > NB ? NA : NB;
  uint32_t b[NB][4];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    if (TR) ldsm_t(b[i], addr + i * plane);
    else ldsm(b[i], addr + i * plane);
  }
#pragma unroll
  for (int s = N - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i <= s; ++i)
      if (i < NA && s - i < NB) {
        mma(d0, a[i], b[s - i][0], b[s - i][1]);
        mma(d1, a[i], b[s - i][2], b[s - i][3]);
      }
}
// The A operand of the 16 x 16 block stored [k][m] at block_at's address.
__device__ __forceinline__ void a_from_t(uint32_t (&a)[4], uint32_t addr) {
  uint32_t r[4];
  ldsm_t(r, addr);
  a[0] = r[0]; a[1] = r[2]; a[2] = r[1]; a[3] = r[3];
}
template <int N>
__device__ __forceinline__ void zero(float (&a)[N][4]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) a[i][j] = 0.f;
}
// mma_pair from zero, added with one rounding to nearest: the tensor cores' sums truncate,
// and a result is a sum of up to a dozen such steps (dk was off by 1.1e-6 of its norm
// without that, by 3.3e-7 with it).
template <int NA, int NB, bool TR>
__device__ __forceinline__ void mma_apart(float (&d0)[4], float (&d1)[4],
                                          const uint32_t (&a)[NA][4], uint32_t addr,
                                          uint32_t plane) {
  float x[2][4];
  zero(x);
  mma_pair<NA, NB, TR>(x[0], x[1], a, addr, plane);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    d0[i] += x[0][i];
    d1[i] += x[1][i];
  }
}

// ------------------------------------------------------------------ loads
__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
// ROWS rows of a tile of W columns as three planes, `plane` bytes apart: row r is
// src + r * ld for r < rows, columns below cols; zeros elsewhere (wide: rows lie on
// 16 bytes).
template <int W, int ROWS>
__device__ __forceinline__ void load_tile(uint32_t dst, uint32_t plane, const float* src,
                                          int64_t ld, int rows, int cols, int wide, int tid,
                                          int nth) {
  constexpr int U = W / 8;
  for (int i = tid; i < ROWS * U; i += nth) {
    const int r = i / U, u = i % U;
    const uint32_t at = dst + tile_at<W>(r, u);
    const float* p = src + r * ld + u * 8;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
    if (r < rows) {
      if (wide && u * 8 + 8 <= cols) {
        const float4 a = *reinterpret_cast<const float4*>(p);
        const float4 b = *reinterpret_cast<const float4*>(p + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (u * 8 + j < cols) v[j] = p[j];
      }
    }
    uint32_t t[4][3];
#pragma unroll
    for (int j = 0; j < 4; ++j) split2<3>(v[2 * j], v[2 * j + 1], t[j]);
#pragma unroll
    for (int n = 0; n < 3; ++n) sts16(at + n * plane, t[0][n], t[1][n], t[2][n], t[3][n]);
  }
}
// Planes of the workspace (dense rows of `ld` elements, `src_plane` elements
// apart) into tiles of W columns; zeros past `rows` rows or `cols` columns.
template <int W, int ROWS, int NT>
__device__ __forceinline__ void load_planes(uint32_t dst, uint32_t plane, const bf16* src,
                                            int64_t ld, int64_t src_plane, int rows, int cols,
                                            int tid, int nth) {
  constexpr int U = W / 8;
  for (int i = tid; i < NT * ROWS * U; i += nth) {
    const int n = i / (ROWS * U), j = i % (ROWS * U), r = j / U, u = j % U;
    const bool in = r < rows && u * 8 < cols;
    cp16(dst + n * plane + tile_at<W>(r, u), in ? src + n * src_plane + r * ld + u * 8 : src,
         in ? 16 : 0);
  }
}
// A value of a tile of TI planes.
template <int W, int TI>
__device__ __forceinline__ float2 tile_pair(const unsigned char* base, uint32_t plane, int row,
                                            int col) {
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = TI - 1; i >= 0; --i) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(
        base + i * plane + tile_at<W>(row, col >> 3) + (col & 7) * 2);
    s.x += lo_of(w);
    s.y += hi_of(w);
  }
  return s;
}

// ------------------------------------------------------------------ launches
// (each returns the launch's error; the first four: fp32)
cudaError_t launch_prepare(const Args& a, cudaStream_t st);
// out (a backward that runs the forward again) and final may be null; S0 and X are written
// where they are given
cudaError_t launch_forward(const Args& a, cudaStream_t st);
cudaError_t launch_reverse(const Args& a, cudaStream_t st);
cudaError_t launch_grads(const Args& a, cudaStream_t st);
// dq and dk of heads that share them: sums of dq_part and dk_part
template <typename T> cudaError_t launch_group_sum(const Args& a, cudaStream_t st);

}  // namespace delta
}  // namespace ssd
