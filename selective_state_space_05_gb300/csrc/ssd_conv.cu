// The causal depthwise conv1d's backward and its one-token step (the forward
// is in ssd_block.cu).  With pre[t] = bias + sum_k w[k] x[t-W+1+k] and
// dpre[t] = dout[t] act'(pre[t]), taps outside the sequence or in another
// document (seq_idx) being zero:
//   dx[s] = sum_k w[k] dpre[s+W-1-k],  dw[k] = sum_t dpre[t] x[t-W+1+k],
//   dbias = sum_t dpre[t]
// Bound by HBM: x and dout are read once and dx is written once.  One thread
// walks a range of tokens of four channels with the filter, the last W inputs
// and the W unfinished dx in registers (rings with compile-time slots: the
// walk is unrolled W times); pre is
// recomputed from the inputs, which are read anyway.  A range reads W-1 tokens
// of its neighbours on either side.  The filter's gradient is summed over the
// range in registers, written once per range and joined by
// launch_column_sum in a fixed order.
//
// Measured on one GB300: 8 x 4096 tokens of 5376 channels, width 4, bf16, 287 us
// with documents and 247 without (3.7 and 4.3 TB/s), where it issues 63 % of the
// cycles on 13 warps an SM (packed fp32x2 instructions were no faster); the same
// in fp32 5.9 TB/s.
#include <stdio.h>

#include <algorithm>

#include "../../include/ssd_block.h"
#include "ssd_common.cuh"
#include "ssd_row.cuh"

namespace ssd {
namespace conv {

constexpr int kMaxW = 8;
constexpr int kCh = 4;          // channels a thread
constexpr int kThreads = 128;
constexpr int kMinRange = 32;   // tokens: the halo of W-1 on either side stays small
constexpr int kCtasPerSm = 5, kCtasPerSmSeq = 4;   // that registers leave room for

struct Raw4 {   // one token's kCh channels as loaded
  uint4 v;
};
__device__ __forceinline__ void raw4(const float* p, Raw4& r) {
  r.v = *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void raw4(const __nv_bfloat16* p, Raw4& r) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  r.v.x = u.x;
  r.v.y = u.y;
}
__device__ __forceinline__ void val4(const Raw4& r, const float*, float (&v)[kCh]) {
  v[0] = __uint_as_float(r.v.x); v[1] = __uint_as_float(r.v.y);
  v[2] = __uint_as_float(r.v.z); v[3] = __uint_as_float(r.v.w);
}
__device__ __forceinline__ void val4(const Raw4& r, const __nv_bfloat16*, float (&v)[kCh]) {
  v[0] = __uint_as_float(r.v.x << 16); v[1] = __uint_as_float(r.v.x & 0xFFFF0000u);
  v[2] = __uint_as_float(r.v.y << 16); v[3] = __uint_as_float(r.v.y & 0xFFFF0000u);
}
__device__ __forceinline__ void put4(float* p, const float (&v)[kCh]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void put4(__nv_bfloat16* p, const float (&v)[kCh]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}

// Asynchronous copy of one token's kCh channels into this thread's own place in
// shared memory (8 bytes of bf16, 16 of fp32).
template <int BYTES>
__device__ __forceinline__ void copy_ahead(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "n"(BYTES)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// grid (channel blocks, ranges, batch).  part: [batch * ranges][C * W + C],
// the range's dweight, then its dbias.  SEQ: with seq_idx.
// x and dout of the next kAhead tokens are on their way through shared memory,
// each thread copying and reading its own channels only (no barrier); with the
// loads held in registers instead, W tokens ahead, the warps waited for them
// (4 of 8 stalls).
template <typename T, int W, bool SEQ>
__global__ void __launch_bounds__(kThreads)
    conv_bwd_kernel(const T* __restrict__ x, TokStride sx, const T* __restrict__ dout,
                    TokStride sdo, const float* __restrict__ w, const float* __restrict__ bias,
                    const int32_t* __restrict__ seq_idx, int64_t L, int64_t range, int C, int silu,
                    T* __restrict__ dx, TokStride sdx, float* __restrict__ part) {
  constexpr int kBytes = kCh * sizeof(T);
  constexpr int kAhead = 64 / kBytes * 2;   // 16 or 8 tokens: 32 KB a CTA
  __shared__ alignas(16) unsigned char ring[2][kAhead][kThreads][kBytes];
  const int c0 = (blockIdx.x * kThreads + threadIdx.x) * kCh;
  if (c0 >= C) return;
  const int64_t b = blockIdx.z;
  const int64_t t0 = (int64_t)blockIdx.y * range;
  const int64_t t1 = t0 + range < L ? t0 + range : L;
  const int64_t tend = t1 + W - 1 < L ? t1 + W - 1 : L;   // dx of the last tokens needs these
  const int n = (int)(tend - t0), own = (int)(t1 - t0);
  const T* xb = x + b * sx.b + c0 + t0 * sx.t;
  const T* db = dout + b * sdo.b + c0 + t0 * sdo.t;
  T* dxb = dx + b * sdx.b + c0 + (t0 - (W - 1)) * sdx.t;   // the token finished at step 0
  const int32_t* sq = SEQ ? seq_idx + b * L + t0 : nullptr;
  float wt[W][kCh], bv[kCh], dw[W][kCh], dbv[kCh];
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
    bv[i] = bias ? bias[c0 + i] : 0.f;
    dbv[i] = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      wt[k][i] = w[(c0 + i) * W + k];
      dw[k][i] = 0.f;
    }
  }
  const T *xp = xb, *dp = db;   // of the next token to copy
  auto ahead = [&](int i) {     // token i of the range, if it is one
    if (i < n) {
      copy_ahead<kBytes>(ring[0][i % kAhead][threadIdx.x], xp);
      copy_ahead<kBytes>(ring[1][i % kAhead][threadIdx.x], dp);
      xp += sx.t;
      dp += sdo.t;
    }
    copy_commit();
  };
  for (int i = 0; i < kAhead; ++i) ahead(i);
  // rings: token t0 + n W + u sits in slot u; the W-1 tokens before t0 in
  // slots 1 .. W-1
  float xr[W][kCh], dr[W][kCh];
  int qr[W], qn[W];   // documents of the window, and of the next W tokens
#pragma unroll
  for (int u = 0; u < W; ++u) {
    qr[u] = 0;
#pragma unroll
    for (int i = 0; i < kCh; ++i) xr[u][i] = dr[u][i] = 0.f;
    const int64_t t = t0 - W + u;
    if (u > 0 && t >= 0) {
      Raw4 r;
      raw4(xb + (u - W) * sx.t, r);
      val4(r, (const T*)nullptr, xr[u]);
      if (SEQ) qr[u] = sq[u - W];
    }
    if (SEQ) qn[u] = u < n ? sq[u] : 0;
  }
  for (int tb = 0; tb < n; tb += W) {
#pragma unroll
    for (int u = 0; u < W; ++u) {
      const int t = tb + u;
      if (t < n) {
        copy_wait<kAhead - 1>();
        Raw4 rx, rd;
        raw4(reinterpret_cast<const T*>(ring[0][t % kAhead][threadIdx.x]), rx);
        raw4(reinterpret_cast<const T*>(ring[1][t % kAhead][threadIdx.x]), rd);
        float g[kCh], pre[kCh];
        val4(rx, (const T*)nullptr, xr[u]);
        val4(rd, (const T*)nullptr, g);
        if (SEQ) {
          qr[u] = qn[u];
          qn[u] = t + W < n ? sq[t + W] : 0;
        }
#pragma unroll
        for (int i = 0; i < kCh; ++i) pre[i] = bv[i];
        bool same[W];   // lag j: token t - j is in t's document (or before the sequence, where x = 0)
#pragma unroll
        for (int j = 0; j < W; ++j) {
          same[j] = !SEQ || qr[(u - j + W) % W] == qr[u];
          if (same[j]) {
#pragma unroll
            for (int i = 0; i < kCh; ++i)
              pre[i] = fmaf(wt[W - 1 - j][i], xr[(u - j + W) % W][i], pre[i]);
          }
        }
        if (silu) {
#pragma unroll
          for (int i = 0; i < kCh; ++i) {
            const float s = row::sigmoid<T>(pre[i]);
            g[i] *= fmaf(s * pre[i], 1.f - s, s);
          }
        }
#pragma unroll
        for (int i = 0; i < kCh; ++i) dr[u][i] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) {
          if (same[j]) {
#pragma unroll
            for (int i = 0; i < kCh; ++i)
              dr[(u - j + W) % W][i] = fmaf(wt[W - 1 - j][i], g[i], dr[(u - j + W) % W][i]);
          }
        }
        if (t < own) {   // the tokens after the range are its neighbour's
#pragma unroll
          for (int j = 0; j < W; ++j) {
            if (same[j]) {
#pragma unroll
              for (int i = 0; i < kCh; ++i)
                dw[W - 1 - j][i] = fmaf(g[i], xr[(u - j + W) % W][i], dw[W - 1 - j][i]);
            }
          }
#pragma unroll
          for (int i = 0; i < kCh; ++i) dbv[i] += g[i];
        }
        if (t >= W - 1) put4(dxb, dr[(u + 1) % W]);   // token t - (W-1): no later one reads it
        dxb += sdx.t;
        ahead(t + kAhead);   // into the place just read
      }
    }
  }
  // tokens whose readers end with the sequence
#pragma unroll
  for (int u = 0; u < W; ++u) {
    // the last token of slot u: the largest t < n with t % W == u
    const int t = u + (n - u + W - 1) / W * W - W;
    if (u < n && t < own && t > n - W) put4(dxb + (int64_t)(t - (n - (W - 1))) * sdx.t, dr[u]);
  }
  copy_wait<0>();
  float* p = part + (b * gridDim.y + blockIdx.y) * ((int64_t)C * (W + 1));
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
#pragma unroll
    for (int k = 0; k < W; ++k) p[(int64_t)(c0 + i) * W + k] = dw[k][i];
    p[(int64_t)C * W + c0 + i] = dbv[i];
  }
}

// One token: the window is the state's W-1 inputs and x; the state moves on
// by one.  One thread per kCh channels of a batch row.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads)
    conv_step_kernel(const T* __restrict__ x, int64_t sx, T* __restrict__ state,
                     const float* __restrict__ w, const float* __restrict__ bias, int C, int silu,
                     T* __restrict__ out) {
  const int c0 = (blockIdx.x * kThreads + threadIdx.x) * kCh;
  if (c0 >= C) return;
  const int64_t b = blockIdx.y;
  T* sb = state + b * (W - 1) * C + c0;
  Raw4 r[W];
#pragma unroll
  for (int k = 0; k < W - 1; ++k) raw4(sb + (int64_t)k * C, r[k]);
  raw4(x + b * sx + c0, r[W - 1]);
  float acc[kCh];
#pragma unroll
  for (int i = 0; i < kCh; ++i) acc[i] = bias ? bias[c0 + i] : 0.f;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    float v[kCh];
    val4(r[k], (const T*)nullptr, v);
#pragma unroll
    for (int i = 0; i < kCh; ++i) acc[i] = fmaf(w[(c0 + i) * W + k], v[i], acc[i]);
    if (k > 0) put4(sb + (int64_t)(k - 1) * C, v);   // exact: the values are T's
  }
  if (silu) {
#pragma unroll
    for (int i = 0; i < kCh; ++i) acc[i] *= row::sigmoid<T>(acc[i]);
  }
  put4(out + b * C + c0, acc);
}

int channel_blocks(int C) { return (C / kCh + kThreads - 1) / kThreads; }

// Tokens a range: as many ranges as fill the SMs once or twice, whichever leaves
// fewer places empty (8 x 4096 tokens x 5376 channels with documents: 285 us in
// two rounds, 309 in one of 528 of 608 places), none shorter than kMinRange.
int64_t range_of(int64_t batch, int64_t seqlen, int C, bool seq) {
  const int64_t places = (int64_t)row::sm_count() * (seq ? kCtasPerSmSeq : kCtasPerSm);
  const int64_t per = channel_blocks(C) * batch;   // CTAs of one range
  int64_t want = std::max<int64_t>(1, places / per);
  const int64_t twice = 2 * places / per;
  if (twice * per > 2 * (want * per) + places / 10) want = twice;
  int64_t r = (seqlen + want - 1) / want;
  r = std::max<int64_t>(r, kMinRange);
  return std::max(r, (seqlen + 65534) / 65535);
}
int64_t ranges_of(int64_t batch, int64_t seqlen, int C, bool seq) {
  const int64_t r = range_of(batch, seqlen, C, seq);
  return (seqlen + r - 1) / r;
}

int bad(int code, const char* msg) { return set_error(code, msg); }
int launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return SSD_OK;
  char m[256];
  snprintf(m, sizeof(m), "%s launch: %s", what, cudaGetErrorString(e));
  return set_error(SSD_ERR_CUDA, m);
}
bool al(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check(int64_t batch, int64_t seqlen, int C, int W, ssd_dtype_t dt) {
  if (dt != SSD_DTYPE_F32 && dt != SSD_DTYPE_BF16) return bad(SSD_ERR_ARG, "unknown dtype");
  if (batch < 1 || seqlen < 1 || C < 1 || batch > 65535)
    return bad(SSD_ERR_ARG, "batch (1..65535), seqlen and channels must be >= 1");
  if (C % 8 != 0) return bad(SSD_ERR_UNSUPPORTED, "channels must be a multiple of 8");
  if (W < 1 || W > kMaxW) return bad(SSD_ERR_UNSUPPORTED, "width must be in [1, 8]");
  if (seqlen >= (1LL << 31)) return bad(SSD_ERR_UNSUPPORTED, "seqlen too large");
  return SSD_OK;
}

// every token's vectors stay aligned, and tokens of an output do not overlap
bool bad_stride(const ssd_stride_t& s, int C, size_t e) {
  return s.batch < 0 || s.token < C || (s.batch * (int64_t)e) % 16 != 0 ||
         (s.token * (int64_t)e) % 16 != 0;
}

}  // namespace conv
}  // namespace ssd

using namespace ssd;
using namespace ssd::conv;

#define SSD_CONV_WIDTHS(LAUNCH) \
  switch (width) {              \
    case 1: LAUNCH(1); break;   \
    case 2: LAUNCH(2); break;   \
    case 3: LAUNCH(3); break;   \
    case 4: LAUNCH(4); break;   \
    case 5: LAUNCH(5); break;   \
    case 6: LAUNCH(6); break;   \
    case 7: LAUNCH(7); break;   \
    default: LAUNCH(8); break;  \
  }

extern "C" {

size_t ssd_causal_conv1d_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int channels,
                                             int width) {
  if (check(batch, seqlen, channels, width, SSD_DTYPE_F32) != SSD_OK) return 0;
  const int64_t most = std::max(ranges_of(batch, seqlen, channels, false),
                                ranges_of(batch, seqlen, channels, true));
  const size_t n = (size_t)(batch * most) * channels * (width + 1);
  return (n * sizeof(float) + 255) & ~(size_t)255;
}

int ssd_causal_conv1d_bwd(const void* dout, ssd_stride_t dout_stride, const void* x,
                          ssd_stride_t x_stride, const float* weight, const float* bias,
                          const int32_t* seq_idx, int64_t batch, int64_t seqlen, int channels,
                          int width, int silu, ssd_dtype_t dtype, void* dx,
                          ssd_stride_t dx_stride, float* dweight, float* dbias, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const int c = check(batch, seqlen, channels, width, dtype);
  if (c != SSD_OK) return c;
  if (!dout || !x || !weight || !dx || !dweight || !workspace)
    return bad(SSD_ERR_NULL, "dout, x, weight, dx, dweight and workspace are required");
  if (!al(dout, 16) || !al(x, 16) || !al(dx, 16) || !al(weight, 4) || !al(bias, 4) ||
      !al(seq_idx, 4) || !al(dweight, 4) || !al(dbias, 4) || !al(workspace, 256))
    return bad(SSD_ERR_ALIGN, "x, dout and dx must be 16-byte, workspace 256-byte aligned");
  const size_t e = dtype == SSD_DTYPE_BF16 ? 2 : 4;
  if (bad_stride(x_stride, channels, e) || bad_stride(dout_stride, channels, e) ||
      bad_stride(dx_stride, channels, e))
    return bad(SSD_ERR_ALIGN,
               "strides must be multiples of 16 bytes, the token strides >= channels");
  if (batch > 1 && dx_stride.batch < channels)
    return bad(SSD_ERR_ARG, "dx: batch rows must not overlap");
  if (workspace_bytes < ssd_causal_conv1d_bwd_workspace_bytes(batch, seqlen, channels, width))
    return bad(SSD_ERR_WORKSPACE, "workspace too small");
  const int64_t range = range_of(batch, seqlen, channels, seq_idx != nullptr);
  const int64_t ranges = (seqlen + range - 1) / range;
  const dim3 grid((unsigned)channel_blocks(channels), (unsigned)ranges, (unsigned)batch);
  float* part = static_cast<float*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const TokStride sx = {x_stride.batch, x_stride.token}, sd = {dout_stride.batch, dout_stride.token},
                  so = {dx_stride.batch, dx_stride.token};
#define SSD_CONV_BWD(T, W)                                                                     \
  (seq_idx ? conv_bwd_kernel<T, W, true> : conv_bwd_kernel<T, W, false>)                       \
  <<<grid, kThreads, 0, st>>>(                                                                 \
      static_cast<const T*>(x), sx, static_cast<const T*>(dout), sd, weight, bias, seq_idx,    \
      seqlen, range, channels, silu, static_cast<T*>(dx), so, part)
#define SSD_CONV_BWD_F(W) SSD_CONV_BWD(float, W)
#define SSD_CONV_BWD_B(W) SSD_CONV_BWD(__nv_bfloat16, W)
  if (dtype == SSD_DTYPE_F32) {
    SSD_CONV_WIDTHS(SSD_CONV_BWD_F)
  } else {
    SSD_CONV_WIDTHS(SSD_CONV_BWD_B)
  }
  const int64_t n = (int64_t)channels * width;
  launch_column_sum(part, batch * ranges, n + channels, n, dweight, dbias ? channels : 0, dbias,
                    st);
  return launched("causal_conv1d_bwd");
}

int ssd_causal_conv1d_step(const void* x, int64_t x_row_stride, void* conv_state,
                           const float* weight, const float* bias, int64_t batch, int channels,
                           int width, int silu, ssd_dtype_t dtype, void* out, void* stream) {
  const int c = check(batch, 1, channels, width, dtype);
  if (c != SSD_OK) return c;
  if (!x || !weight || !out || (width > 1 && !conv_state))
    return bad(SSD_ERR_NULL, "x, conv_state, weight and out are required");
  const size_t e = dtype == SSD_DTYPE_BF16 ? 2 : 4;
  if (!al(x, 16) || !al(conv_state, 16) || !al(out, 16) || !al(weight, 4) || !al(bias, 4))
    return bad(SSD_ERR_ALIGN, "x, conv_state and out must be 16-byte aligned");
  if (batch > 1 && (x_row_stride < 0 || (x_row_stride * (int64_t)e) % 16 != 0))
    return bad(SSD_ERR_ALIGN, "x's row stride must be a multiple of 16 bytes");
  const dim3 grid((unsigned)channel_blocks(channels), (unsigned)batch);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
#define SSD_CONV_STEP(T, W)                                                                \
  conv_step_kernel<T, W><<<grid, kThreads, 0, st>>>(                                       \
      static_cast<const T*>(x), x_row_stride, static_cast<T*>(conv_state), weight, bias,   \
      channels, silu, static_cast<T*>(out))
#define SSD_CONV_STEP_F(W) SSD_CONV_STEP(float, W)
#define SSD_CONV_STEP_B(W) SSD_CONV_STEP(__nv_bfloat16, W)
  if (dtype == SSD_DTYPE_F32) {
    SSD_CONV_WIDTHS(SSD_CONV_STEP_F)
  } else {
    SSD_CONV_WIDTHS(SSD_CONV_STEP_B)
  }
  return launched("causal_conv1d_step");
}

}  // extern "C"
