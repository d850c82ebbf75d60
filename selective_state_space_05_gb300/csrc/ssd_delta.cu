// C ABI of the gated delta rule (include/ssd_delta.h): checks, workspace, the
// launch sequence and the one-token step.
#include <math.h>
#include <stdio.h>

#include <mutex>

#include "../../include/ssd_delta.h"
#include "ssd_delta_tc.cuh"
#include "ssd_row.cuh"

namespace ssd {
namespace delta {
namespace {

int bad(int code, const char* msg) { return set_error(code, msg); }
int cuda_bad(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return SSD_OK;
  char m[256];
  snprintf(m, sizeof(m), "%s: %s", where, cudaGetErrorString(e));
  return set_error(SSD_ERR_CUDA, m);
}
bool off(const void* p, size_t align) { return ((uintptr_t)p & (align - 1)) != 0; }
size_t up(size_t v) { return (v + 255) & ~(size_t)255; }

constexpr int kMaxHeaddim = 2048;

int check_sizes(int64_t B, int64_t L, int H, int V, int K, int G, int dtype) {
  if (dtype != SSD_DTYPE_F32 && dtype != SSD_DTYPE_BF16) return bad(SSD_ERR_ARG, "unknown dtype");
  if (B < 1 || L < 1 || H < 1 || V < 1 || K < 1 || G < 1)
    return bad(SSD_ERR_ARG, "batch, seqlen, nheads, headdim, dstate and ngroups must be >= 1");
  if (H % G) return bad(SSD_ERR_ARG, "nheads must be a multiple of ngroups");
  if (K > 128) return bad(SSD_ERR_UNSUPPORTED, "dstate must be at most 128");
  if (V > kMaxHeaddim) return bad(SSD_ERR_UNSUPPORTED, "headdim must be at most 2048");
  const int C = dtype == SSD_DTYPE_BF16 ? Mode<bf16>::C : Mode<float>::C;
  if (B > 0x7fffffffLL || L > (1LL << 40) ||
      (double)B * H * ((double)(L + C - 1) / C) >= 2147483648.0)
    return bad(SSD_ERR_UNSUPPORTED, "batch * nheads * chunks must be below 2^31");
  return SSD_OK;
}

Args sizes(int64_t B, int64_t L, int H, int V, int K, int G, int dtype) {
  Args a = {};
  const int C = dtype == SSD_DTYPE_BF16 ? Mode<bf16>::C : Mode<float>::C;
  a.L = L;
  a.B = (int)B;
  a.H = H;
  a.G = G;
  a.K = K;
  a.V = V;
  a.nc = (int)((L + C - 1) / C);
  a.KP = K <= 64 ? 64 : 128;
  a.tc = dtype == SSD_DTYPE_BF16;
  a.VP = a.tc ? (V + 127) / 128 * 128 : (V + 15) / 16 * 16;
  // Segments one after another only where there are more sequences than SMs: eight or so for
  // each SM's share (a segment costs the state's way through the L2, about the time of a
  // chunk), at least eight chunks long.  Measured: 320 sequences of 64 chunks in whole 863
  // us, in segments 800; with as many as SMs or fewer every one has its own SM.
  a.segs = 1;
  a.seg = a.nc;
  const int64_t lanes = (int64_t)a.B * H * (a.VP / 128), sms = row::sm_count();
  if (a.tc && lanes > sms) {
    const int64_t share = lanes * a.nc / sms;
    int64_t seg = share / 8 > 8 ? share / 8 : 8;
    if (seg < a.nc) {
      a.seg = (int)seg;
      a.segs = (int)((a.nc + seg - 1) / seg);
    }
  }
  a.pass = kWhole;
  a.qcols = a.kcols = K;
  a.vcols = a.docols = V;
  return a;
}

// The tcgen05 kernels read rows by tensor maps: on 16 bytes, strides above 0.
// Others are first copied to dense rows of a multiple of eight columns.
int up8(int n) { return (n + 7) & ~7; }
size_t packed_bytes(const Args& a, int rows, int cols) {
  return up((size_t)a.B * a.L * rows * up8(cols) * 2);
}
__global__ void __launch_bounds__(256)
    pack_kernel(const bf16* __restrict__ src, TokStride s, int64_t L, int64_t n, int rows, int cols,
                int wide, bf16* __restrict__ dst) {
  const int64_t total = n * rows * wide;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int c = (int)(i % wide);
    const int64_t r = i / wide % rows, t = i / wide / rows;
    dst[i] = c < cols ? src[toff(s, t / L, t % L) + r * cols + c] : __float2bfloat16_rn(0.f);
  }
}
cudaError_t pack(const Args& a, const void** src, TokStride* s, int* ncols, int rows, char* to,
                 cudaStream_t st) {
  const int cols = *ncols, wide = up8(cols);
  const int64_t n = (int64_t)a.B * a.L, ctas = (n * rows * wide + 255) / 256;
  pack_kernel<<<(unsigned)(ctas < 16384 ? ctas : 16384), 256, 0, st>>>(
      static_cast<const bf16*>(*src), *s, a.L, n, rows, cols, wide, reinterpret_cast<bf16*>(to));
  *src = to;
  *s = {a.L * rows * wide, (int64_t)rows * wide};
  *ncols = wide;
  return cudaGetLastError();
}

size_t state_bytes(const Args& a) { return (size_t)a.B * a.H * a.V * a.K * 4; }

template <typename F>
void carve_work(Args& a, F take) {
  if (!a.tc) return;
  const size_t lanes = (size_t)a.B * a.H * (a.VP / 128);
  const size_t slots = a.pass == kParts ? lanes * (a.segs - 1) + (size_t)a.B * a.H * (a.segs - 2)
                       : a.segs > 1     ? lanes
                                        : 0;
  a.ctrl = reinterpret_cast<int*>(take((1 + lanes) * sizeof(int)));
  a.slots = reinterpret_cast<float*>(take(slots * 128 * a.KP * 4));
  a.first = reinterpret_cast<float*>(take(a.pass == kParts ? state_bytes(a) : 0));
}
// A few long sequences leave most SMs idle: their segments run all at once, in two
// passes, where that takes fewer chunks' time than the sequence has chunks.  The first
// pass has 2 segs - 3 items a sequence (of 128 channels), the second segs; an item takes
// three chunks' time to start, joining one a segment, two launches eight.  Measured: 512
// chunks of 16 heads in one pass 1.56 ms, in two of 6 segments 0.63, of 19 (no time to
// start counted) 0.70; 16 chunks stay in one pass.
void split(Args& a) {
  const int64_t lanes = (int64_t)a.B * a.H * (a.VP / 128), heads = (int64_t)a.B * a.H;
  const int64_t sms = row::sm_count();
  if (!a.tc || a.segs > 1 || lanes >= sms) return;
  int64_t best = a.nc;
  for (int64_t segs = 2; segs <= 64 && segs * 8 <= a.nc; ++segs) {
    const int64_t seg = (a.nc + segs - 1) / segs, n = (a.nc + seg - 1) / seg;
    const int64_t first = lanes * (n - 1) + heads * (n - 2), second = lanes * n;
    const int64_t steps = ((first + sms - 1) / sms + (second + sms - 1) / sms) * (seg + 3) + n + 8;
    if (steps < best) {
      best = steps;
      a.seg = (int)seg;
      a.segs = (int)n;
      a.pass = kParts;
    }
  }
}

// The forward's pieces of a workspace at `base`, and how many bytes they take.
template <typename T>
size_t carve(Args& a, void* base, bool keep) {   // (the forward's `a`: split)
  constexpr int C = Mode<T>::C, NT = Mode<T>::NT;
  const size_t n = (size_t)a.B * a.H * a.nc;
  char* p = static_cast<char*>(base);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* r = p + at;
    at += up(bytes);
    return r;
  };
  a.T = a.P = a.S0 = a.X = nullptr;
  a.vec = nullptr;
  a.T = reinterpret_cast<bf16*>(take(n * NT * C * C * 2 * (a.tc ? 2 : 1)));   // (P beside T)
  if (!a.tc) a.P = reinterpret_cast<bf16*>(take(n * NT * C * C * 2));
  carve_work(a, take);
  a.vec = reinterpret_cast<float*>(take(n * vec_floats<C>() * 4));
  if (keep) {
    a.S0 = reinterpret_cast<bf16*>(take(n * NT * a.VP * a.KP * 2));
    a.X = reinterpret_cast<bf16*>(take(n * NT * C * a.VP * 2));
  }
  return at;
}
// The backward's own.
template <typename T>
size_t carve_bwd(Args& a, void* base) {
  constexpr int C = Mode<T>::C, NT = Mode<T>::NT;
  const size_t n = (size_t)a.B * a.H * a.nc;
  char* p = static_cast<char*>(base);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* r = p + at;
    at += up(bytes);
    return r;
  };
  a.dS = reinterpret_cast<bf16*>(take(n * NT * a.VP * a.KP * 2));
  a.dY = reinterpret_cast<bf16*>(take(n * NT * C * a.VP * 2));
  carve_work(a, take);
  a.dq_part = a.dk_part = nullptr;
  if (a.H != a.G) {
    a.dq_part = reinterpret_cast<float*>(take((size_t)a.B * a.L * a.H * a.K * 4));
    a.dk_part = reinterpret_cast<float*>(take((size_t)a.B * a.L * a.H * a.K * 4));
  }
  return at;
}
size_t fwd_bytes(Args& a, int dtype, void* base, bool keep) {
  split(a);
  return dtype == SSD_DTYPE_BF16 ? carve<bf16>(a, base, keep) : carve<float>(a, base, keep);
}
size_t bwd_bytes(Args& a, int dtype, void* base) {
  split(a);
  return dtype == SSD_DTYPE_BF16 ? carve_bwd<bf16>(a, base) : carve_bwd<float>(a, base);
}

bool bad_stride(ssd_stride_t s) {
  return s.batch < 0 || s.token < 0 || s.batch > (1LL << 40) || s.token > (1LL << 40);
}
// Whether a tensor map takes such rows (a stride of 0 only along a length of 1).
bool mapped(const Args& a, int wide, TokStride s) {
  const int64_t most = 1LL << 38;
  return wide && (s.t > 0 || a.L == 1) && (s.b > 0 || a.B == 1) && s.t <= most && s.b <= most;
}
// Whether rows of `n` elements at these strides lie on 16 bytes.
int wide_rows(const void* p, ssd_stride_t s, int n, int esize) {
  return !off(p, 16) && (s.batch * esize) % 16 == 0 && (s.token * esize) % 16 == 0 &&
         (n * esize) % 16 == 0;
}

int fill_inputs(Args& a, const void* q, ssd_stride_t sq, const void* k, ssd_stride_t sk,
                const void* v, ssd_stride_t sv, const float* g, const float* beta, float scale,
                const float* init, const int32_t* seq, int dtype) {
  const int es = dtype == SSD_DTYPE_BF16 ? 2 : 4;
  if (!q || !k || !v || !g || !beta) return bad(SSD_ERR_NULL, "q, k, v, g and beta are required");
  if (bad_stride(sq) || bad_stride(sk) || bad_stride(sv))
    return bad(SSD_ERR_ARG, "strides must be in [0, 2^40]");
  if (!(fabsf(scale) <= 3.0e38f)) return bad(SSD_ERR_ARG, "scale must be finite");
  if (off(q, es) || off(k, es) || off(v, es) || off(g, 4) || off(beta, 4) || off(init, 4) ||
      off(seq, 4))
    return bad(SSD_ERR_ALIGN, "a pointer is not aligned to its element");
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.scale = scale;
  a.init = init;
  a.seq = seq;
  a.sq = {sq.batch, sq.token};
  a.sk = {sk.batch, sk.token};
  a.sv = {sv.batch, sv.token};
  a.wide_q = wide_rows(q, sq, a.K, es);
  a.wide_k = wide_rows(k, sk, a.K, es);
  a.wide_v = wide_rows(v, sv, a.V, es);
  return SSD_OK;
}

cudaError_t run_forward(const Args& a, cudaStream_t st) {
  if (a.tc) {
    const cudaError_t e = launch_tc_prepare(a, st);
    return e != cudaSuccess ? e : launch_tc_forward(a, st);
  }
  const cudaError_t e = launch_prepare(a, st);
  return e != cudaSuccess ? e : launch_forward(a, st);
}

bool inputs_mapped(const Args& a) {
  return mapped(a, a.wide_q, a.sq) && mapped(a, a.wide_k, a.sk) && mapped(a, a.wide_v, a.sv);
}
size_t pack_bytes(const Args& a, bool aligned) {
  return !a.tc || aligned
             ? 0
             : 2 * packed_bytes(a, a.G, a.K) + packed_bytes(a, a.H, a.V);
}
size_t pack_dout_bytes(const Args& a) { return a.tc ? packed_bytes(a, a.H, a.V) : 0; }
// Copies q, k and v where they are not mapped, to pack_bytes at `at`.
cudaError_t pack_inputs(Args& a, char* at, cudaStream_t st) {
  if (!a.tc || inputs_mapped(a)) return cudaSuccess;
  const size_t n = packed_bytes(a, a.G, a.K);
  cudaError_t e = pack(a, &a.q, &a.sq, &a.qcols, a.G, at, st);
  if (e == cudaSuccess) e = pack(a, &a.k, &a.sk, &a.kcols, a.G, at + n, st);
  if (e == cudaSuccess) e = pack(a, &a.v, &a.sv, &a.vcols, a.H, at + 2 * n, st);
  return e;
}

// Memory that a call reads or writes.
struct Span {
  const void* p;
  unsigned __int128 n;   // bytes
};
Span dense(const void* p, int64_t n, int size) { return {p, (unsigned __int128)n * size}; }
Span tokens(const void* p, ssd_stride_t s, int64_t B, int64_t L, int64_t n, int size) {
  return {p, ((unsigned __int128)(B - 1) * s.batch + (unsigned __int128)(L - 1) * s.token + n) * size};
}
bool meet(Span a, Span b) {
  return a.p && b.p && (uintptr_t)a.p < (uintptr_t)b.p + b.n && (uintptr_t)b.p < (uintptr_t)a.p + a.n;
}
// Whether one of the outputs meets an input or another output.
template <int NO, int NI>
bool any_meet(const Span (&out)[NO], const Span (&in)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return true;
    for (const Span& x : in)
      if (meet(out[i], x)) return true;
  }
  return false;
}

// One token.  HBM-bound on the fp32 state, read and written once.  A warp takes
// kRows rows of a head's state, all their loads in flight before the first is
// used; with a = S q and b = S k of the old state, u = beta (v - e^g b) and
// out = scale (e^g a + u (k q)), so that both row sums come from one pass.  320 states
// of 128 x 128: 10.0 us from a cold L2, 4.2 TB/s; eight of 64 x 64: 4.9 us, the latency
// of a launch and of one load after another.
constexpr int kStepWarps = 4, kRows = 8;

template <typename T, bool VEC>
__global__ void __launch_bounds__(kStepWarps * 32)
    step_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                const float* __restrict__ g, const float* __restrict__ beta, float scale,
                float* __restrict__ state, int H, int V, int K, int G, T* __restrict__ out) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t bh = blockIdx.x;
  const int h = (int)(bh % H);
  const int64_t at = (bh / H * G + h / (H / G)) * K;
  // this lane's four columns: neighbours where rows are whole float4s
  float kv[4], qv[4];
  int col[4];
  float kq = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    col[j] = VEC ? lane * 4 + j : lane + 32 * j;
    kv[j] = col[j] < K ? to_f(k[at + col[j]]) : 0.f;
    qv[j] = col[j] < K ? to_f(q[at + col[j]]) : 0.f;
    kq = fmaf(kv[j], qv[j], kq);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, o);
  const float decay = expf(g[bh]), be = beta[bh];
  const int v0 = (blockIdx.y * kStepWarps + warp) * kRows;
  if (v0 >= V) return;
  float* const S = state + (bh * V + v0) * K;
  float s[kRows][4];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const bool row = v0 + r < V;
    if (VEC) {
      float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row && col[0] < K) w = *reinterpret_cast<const float4*>(S + (int64_t)r * K + col[0]);
      s[r][0] = w.x; s[r][1] = w.y; s[r][2] = w.z; s[r][3] = w.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) s[r][j] = row && col[j] < K ? S[(int64_t)r * K + col[j]] : 0.f;
    }
  }
  float vv[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) vv[r] = v0 + r < V ? to_f(v[bh * V + v0 + r]) : 0.f;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    float sa = 0.f, sb = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[r][j] *= decay;
      sa = fmaf(s[r][j], qv[j], sa);
      sb = fmaf(s[r][j], kv[j], sb);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sa += __shfl_xor_sync(0xffffffffu, sa, o);
      sb += __shfl_xor_sync(0xffffffffu, sb, o);
    }
    const float u = be * (vv[r] - sb);
#pragma unroll
    for (int j = 0; j < 4; ++j) s[r][j] = fmaf(u, kv[j], s[r][j]);
    if (v0 + r >= V) continue;
    if (lane == r) out[bh * V + v0 + r] = from_f<T>(scale * fmaf(u, kq, sa));
    if (VEC) {
      if (col[0] < K)
        *reinterpret_cast<float4*>(S + (int64_t)r * K + col[0]) =
            make_float4(s[r][0], s[r][1], s[r][2], s[r][3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col[j] < K) S[(int64_t)r * K + col[j]] = s[r][j];
    }
  }
}

template <typename T>
cudaError_t run_step(const void* q, const void* k, const void* v, const float* g,
                     const float* beta, float scale, float* state, int64_t B, int H, int V, int K,
                     int G, void* out, cudaStream_t st) {
  const dim3 grid((unsigned)(B * H), (unsigned)((V + kStepWarps * kRows - 1) / (kStepWarps * kRows)));
  const T *qt = static_cast<const T*>(q), *kt = static_cast<const T*>(k),
          *vt = static_cast<const T*>(v);
  if (K % 4 == 0 && !off(state, 16))
    step_kernel<T, true><<<grid, kStepWarps * 32, 0, st>>>(qt, kt, vt, g, beta, scale, state, H, V,
                                                           K, G, static_cast<T*>(out));
  else
    step_kernel<T, false><<<grid, kStepWarps * 32, 0, st>>>(qt, kt, vt, g, beta, scale, state, H,
                                                            V, K, G, static_cast<T*>(out));
  return cudaGetLastError();
}

}  // namespace

namespace {
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
}  // namespace

int status(int reset, cudaStream_t st, int* bits) {
  int (*const words[])(int, cudaStream_t, int*) = {tc_prepare_status, tc_forward_status,
                                                   tc_reverse_status, tc_grads_status};
  int e = 0;
  *bits = 0;
  for (auto w : words) {
    int now = 0;
    if (e == 0) e = w(reset, st, &now);
    *bits |= now;
  }
  return e;
}

cudaError_t copy_first(const Args& a, const float** from, const float* to, cudaStream_t st) {
  if (!to || *from != to) return cudaSuccess;
  const cudaError_t e =
      cudaMemcpyAsync(a.first, *from, state_bytes(a), cudaMemcpyDeviceToDevice, st);
  *from = a.first;
  return e;
}

cudaError_t start_work(const Args& a, int* grid, cudaStream_t st) {
  const int lanes = a.B * a.H * (a.VP / 128), sms = row::sm_count();
  const int items = a.pass == kParts ? lanes * (a.segs - 1) + a.B * a.H * (a.segs - 2)
                    : a.pass == kJoined ? lanes * a.segs
                                        : lanes;
  *grid = items < sms ? items : sms;
  return cudaMemsetAsync(a.ctrl, 0, (1 + lanes) * sizeof(int), st);
}

bool token_map(CUtensorMap* m, const void* base, int cols, int rows, int64_t L, int B, TokStride s,
               bool swizzle) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[4] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)L, (cuuint64_t)B};
  // (a stride along a length of 1 is never walked)
  cuuint64_t strides[3] = {(cuuint64_t)cols * 2, (cuuint64_t)(s.t > 0 ? s.t : cols) * 2,
                           (cuuint64_t)(s.b > 0 ? s.b : cols) * 2};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)kC, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace delta
}  // namespace ssd

using namespace ssd::delta;

extern "C" {

int ssd_delta_abi_version(void) { return SSD_DELTA_ABI_VERSION; }

size_t ssd_delta_scan_workspace_bytes(int64_t batch, int64_t seqlen, int nheads, int headdim,
                                      int dstate, int ngroups, ssd_dtype_t dtype, int keep, int aligned) {
  if (check_sizes(batch, seqlen, nheads, headdim, dstate, ngroups, dtype) != SSD_OK) return 0;
  Args a = sizes(batch, seqlen, nheads, headdim, dstate, ngroups, dtype);
  const size_t n = fwd_bytes(a, dtype, nullptr, keep != 0) + pack_bytes(a, aligned != 0);
  return n ? n : 256;
}

int ssd_delta_scan_fwd(const void* q, ssd_stride_t q_stride, const void* k, ssd_stride_t k_stride,
                       const void* v, ssd_stride_t v_stride, const float* g, const float* beta,
                       float scale, const float* initial_states, const int32_t* seq_idx,
                       int64_t batch, int64_t seqlen, int nheads, int headdim, int dstate,
                       int ngroups, ssd_dtype_t dtype, void* out, float* final_states, int keep,
                       void* workspace, size_t workspace_bytes, void* stream) {
  int c = check_sizes(batch, seqlen, nheads, headdim, dstate, ngroups, dtype);
  if (c != SSD_OK) return c;
  Args a = sizes(batch, seqlen, nheads, headdim, dstate, ngroups, dtype);
  c = fill_inputs(a, q, q_stride, k, k_stride, v, v_stride, g, beta, scale, initial_states,
                  seq_idx, dtype);
  if (c != SSD_OK) return c;
  if (!out || !workspace) return bad(SSD_ERR_NULL, "out and workspace are required");
  if (off(out, dtype == SSD_DTYPE_BF16 ? 2 : 4) || off(final_states, 4))
    return bad(SSD_ERR_ALIGN, "a pointer is not aligned to its element");
  if (off(workspace, 256)) return bad(SSD_ERR_ALIGN, "workspace must be 256-byte aligned");
  const size_t kept = fwd_bytes(a, dtype, workspace, keep != 0);
  const size_t used = kept + pack_bytes(a, inputs_mapped(a));
  if (workspace_bytes < used)
    return bad(SSD_ERR_WORKSPACE, "workspace too small");
  const int es = dtype == SSD_DTYPE_BF16 ? 2 : 4;
  const int64_t hs = batch * seqlen * nheads, states = batch * nheads * headdim * dstate;
  const Span outs[] = {dense(out, hs * headdim, es), dense(final_states, states, 4),
                       dense(workspace, (int64_t)used, 1)};
  const Span ins[] = {tokens(q, q_stride, batch, seqlen, (int64_t)ngroups * dstate, es),
                      tokens(k, k_stride, batch, seqlen, (int64_t)ngroups * dstate, es),
                      tokens(v, v_stride, batch, seqlen, (int64_t)nheads * headdim, es),
                      dense(g, hs, 4), dense(beta, hs, 4), dense(seq_idx, batch * seqlen, 4),
                      dense(initial_states == final_states ? nullptr : initial_states, states, 4)};
  if (any_meet(outs, ins))
    return bad(SSD_ERR_ARG, "an output overlaps an input or another output "
                            "(final_states may be initial_states)");
  a.out = out;
  a.wide_out = wide_rows(out, {0, 0}, headdim, dtype == SSD_DTYPE_BF16 ? 2 : 4);
  a.final = final_states;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = pack_inputs(a, static_cast<char*>(workspace) + kept, st);
  if (e == cudaSuccess) e = run_forward(a, st);
  return cuda_bad(e, "delta_scan_fwd launch");
}

size_t ssd_delta_scan_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int nheads, int headdim,
                                          int dstate, int ngroups, ssd_dtype_t dtype, int saved, int aligned) {
  if (check_sizes(batch, seqlen, nheads, headdim, dstate, ngroups, dtype) != SSD_OK) return 0;
  Args a = sizes(batch, seqlen, nheads, headdim, dstate, ngroups, dtype);
  Args f = a;
  return bwd_bytes(a, dtype, nullptr) + (saved ? 0 : fwd_bytes(f, dtype, nullptr, true)) +
         (aligned ? 0 : pack_bytes(a, false) + pack_dout_bytes(a));
}

int ssd_delta_scan_bwd(const void* dout, const float* dfinal_states, const void* q,
                       ssd_stride_t q_stride, const void* k, ssd_stride_t k_stride, const void* v,
                       ssd_stride_t v_stride, const float* g, const float* beta, float scale,
                       const float* initial_states, const int32_t* seq_idx, int64_t batch,
                       int64_t seqlen, int nheads, int headdim, int dstate, int ngroups,
                       ssd_dtype_t dtype, const void* saved, size_t saved_bytes, void* dq, void* dk,
                       void* dv, float* dg, float* dbeta, float* d_initial_states, void* workspace,
                       size_t workspace_bytes, void* stream) {
  int c = check_sizes(batch, seqlen, nheads, headdim, dstate, ngroups, dtype);
  if (c != SSD_OK) return c;
  Args a = sizes(batch, seqlen, nheads, headdim, dstate, ngroups, dtype);
  c = fill_inputs(a, q, q_stride, k, k_stride, v, v_stride, g, beta, scale, initial_states,
                  seq_idx, dtype);
  if (c != SSD_OK) return c;
  if (!dout || !dq || !dk || !dv || !dg || !dbeta || !workspace)
    return bad(SSD_ERR_NULL, "dout, dq, dk, dv, dg, dbeta and workspace are required");
  const int es = dtype == SSD_DTYPE_BF16 ? 2 : 4;
  if (off(dout, es) || off(dv, es) || off(dq, 2 * es) || off(dk, 2 * es) || off(dg, 4) ||
      off(dbeta, 4) || off(dfinal_states, 4) || off(d_initial_states, 4))
    return bad(SSD_ERR_ALIGN, "a pointer is not aligned to its element (dq, dk: to two)");
  if (off(workspace, 256) || off(saved, 256))
    return bad(SSD_ERR_ALIGN, "workspace and saved must be 256-byte aligned");
  Args f = a;   // the forward's pieces, and its work where it is computed again
  const size_t kept = fwd_bytes(f, dtype, nullptr, true), own = bwd_bytes(a, dtype, nullptr);
  if (saved && saved_bytes < kept)
    return bad(SSD_ERR_WORKSPACE, "saved is not the workspace of a forward with keep at these sizes");
  const int64_t hv = (int64_t)nheads * headdim;
  a.dout = dout;
  a.sdo = {seqlen * hv, hv};
  a.wide_do = wide_rows(dout, {0, 0}, headdim, es);
  const bool aligned = inputs_mapped(a) && a.wide_do;
  const size_t used = own + (saved ? 0 : kept);
  const size_t need = used + (aligned ? 0 : pack_bytes(a, false) + pack_dout_bytes(a));
  if (workspace_bytes < need)
    return bad(SSD_ERR_WORKSPACE, "workspace too small");
  const int64_t rows = batch * seqlen, states = batch * nheads * headdim * dstate;
  const int64_t gk = (int64_t)ngroups * dstate;
  const Span outs[] = {dense(dq, rows * gk, es), dense(dk, rows * gk, es), dense(dv, rows * hv, es),
                       dense(dg, rows * nheads, 4), dense(dbeta, rows * nheads, 4),
                       dense(d_initial_states, states, 4), dense(workspace, (int64_t)need, 1)};
  const Span ins[] = {tokens(q, q_stride, batch, seqlen, gk, es),
                      tokens(k, k_stride, batch, seqlen, gk, es),
                      tokens(v, v_stride, batch, seqlen, hv, es), dense(dout, rows * hv, es),
                      dense(g, rows * nheads, 4), dense(beta, rows * nheads, 4),
                      dense(seq_idx, rows, 4), dense(initial_states, states, 4),
                      dense(saved, (int64_t)kept, 1),
                      dense(dfinal_states == d_initial_states ? nullptr : dfinal_states, states, 4)};
  if (any_meet(outs, ins))
    return bad(SSD_ERR_ARG, "an output overlaps an input or another output "
                            "(d_initial_states may be dfinal_states)");
  fwd_bytes(f, dtype, saved ? const_cast<void*>(saved) : static_cast<char*>(workspace) + own, true);
  bwd_bytes(a, dtype, workspace);
  a.T = f.T;
  a.P = f.P;
  a.vec = f.vec;
  a.S0 = f.S0;
  a.X = f.X;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* const at = static_cast<char*>(workspace) + used;
  cudaError_t e = pack_inputs(a, at, st);
  if (e == cudaSuccess && a.tc && !a.wide_do)
    e = pack(a, &a.dout, &a.sdo, &a.docols, a.H, at + pack_bytes(a, false), st);
  if (e == cudaSuccess && !saved) {
    f.q = a.q;
    f.k = a.k;
    f.v = a.v;
    f.sq = a.sq;
    f.sk = a.sk;
    f.sv = a.sv;
    f.qcols = a.qcols;
    f.kcols = a.kcols;
    f.vcols = a.vcols;
    e = run_forward(f, st);
  }
  a.dfinal = dfinal_states;
  a.dinit = d_initial_states;
  a.dv = dv;
  a.wide_dv = wide_rows(dv, {0, 0}, headdim, es);
  a.dq = dq;
  a.dk = dk;
  a.dg = dg;
  a.dbeta = dbeta;
  if (a.tc) {
    if (e == cudaSuccess) e = launch_tc_reverse(a, st);
    if (e == cudaSuccess) e = launch_tc_grads(a, st);
  } else {
    if (e == cudaSuccess) e = launch_reverse(a, st);
    if (e == cudaSuccess) e = launch_grads(a, st);
  }
  return cuda_bad(e, "delta_scan_bwd launch");
}

int ssd_delta_decode_step(const void* q, const void* k, const void* v, const float* g,
                          const float* beta, float scale, float* state, int64_t batch, int nheads,
                          int headdim, int dstate, int ngroups, ssd_dtype_t dtype, void* out,
                          void* stream) {
  const int c = check_sizes(batch, 1, nheads, headdim, dstate, ngroups, dtype);
  if (c != SSD_OK) return c;
  if (!q || !k || !v || !g || !beta || !state || !out)
    return bad(SSD_ERR_NULL, "q, k, v, g, beta, state and out are required");
  const size_t es = dtype == SSD_DTYPE_BF16 ? 2 : 4;
  if (off(q, es) || off(k, es) || off(v, es) || off(out, es) || off(g, 4) || off(beta, 4) ||
      off(state, 4))
    return bad(SSD_ERR_ALIGN, "a pointer is not aligned to its element");
  if (!(fabsf(scale) <= 3.0e38f)) return bad(SSD_ERR_ARG, "scale must be finite");
  const int64_t hs = batch * nheads, gk = batch * ngroups * dstate;
  const Span outs[] = {dense(out, hs * headdim, (int)es), dense(state, hs * headdim * dstate, 4)};
  const Span ins[] = {dense(q, gk, (int)es), dense(k, gk, (int)es), dense(g, hs, 4),
                      dense(beta, hs, 4), dense(v == out ? nullptr : v, hs * headdim, (int)es)};
  if (any_meet(outs, ins))
    return bad(SSD_ERR_ARG, "out or state overlaps an input or the other (out may be v)");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cuda_bad(dtype == SSD_DTYPE_BF16
                      ? run_step<bf16>(q, k, v, g, beta, scale, state, batch, nheads, headdim,
                                       dstate, ngroups, out, st)
                      : run_step<float>(q, k, v, g, beta, scale, state, batch, nheads, headdim,
                                        dstate, ngroups, out, st),
                  "delta_decode_step launch");
}

}  // extern "C"
