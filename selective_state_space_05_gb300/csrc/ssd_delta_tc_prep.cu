// The tcgen05 path's first launch: the vectors, T and P of all chunks at once, one
// CTA of four warps per (chunk, head, batch row).  k k^T and q k^T and the inverse's
// products run on mma.sync: their operands are 16-row blocks that stay in
// registers from one product to the next, and there are many CTAs an SM to fill the
// time between them.  T's and P's terms go out as swizzled tiles, which the chunks'
// kernels copy as they are.  (As a role of the forward's own CTAs this work was in its
// chunks' way: 1.16 ms for the two against 0.94 apart.)
// 20480 chunks of 128 columns take 277 us for 66 KB each, in and out, 5.0 TB/s: half of it
// is T and P on their way to the chunks' kernels.  Four CTAs an SM: their warps' latency
// counts too (323 us before decays and terms were computed two values an instruction).
#include "ssd_delta_tc.cuh"

namespace ssd {
namespace delta {
namespace prep {

constexpr int kThreads = 128;

template <int KP>
struct Smem {
  union {
    unsigned char kq[KP / 64][2][kTile];   // 64 columns: 64 rows of K, 64 of Q
    unsigned char tp[4][kTile];            // afterwards: T's terms, P's terms
  };
  unsigned char a[2][kTile];               // the inverse's A, two terms
  float diag[4][kDiag];
  alignas(16) float vec[vec_floats<kC>()];
  uint64_t full;
  volatile int gave_up;
};
__device__ int g_status;
std::atomic<bool> g_launched{false};

template <int KP>
__global__ void __launch_bounds__(kThreads, 4)
    tc_prepare_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ Args a) {
  extern __shared__ unsigned char raw[];
  Smem<KP>& s = *reinterpret_cast<Smem<KP>*>(raw + ((1024 - (saddr(raw) & 1023)) & 1023));
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int64_t id = blockIdx.x;               // (b H + h) nc + c
  const int c = (int)(id % a.nc), h = (int)(id / a.nc % a.H), b = (int)(id / a.nc / a.H);
  const int kg = h / (a.H / a.G);
  if (tid == 0) {
    tc::mbar_init(&s.full, 1);
    tc::mbar_fence_init();
    s.gave_up = 0;
    tc::mbar_arrive_expect_tx(&s.full, KP / 64 * 2 * kTile);
    for (int i = 0; i < KP / 64; ++i) {
      tc::tma_load_4d(s.kq[i][0], &mk, &s.full, i * 64, kg, c * kC, b);
      tc::tma_load_4d(s.kq[i][1], &mq, &s.full, i * 64, kg, c * kC, b);
    }
  }
  if (w == 0) chunk_vectors(load_gates(a, b, h, (int64_t)c * kC, lane), s.vec, lane);
  __syncthreads();
  wait_for(&s.full, 0, &s.gave_up, &g_status);
  const bool keys = w < 2;
  const uint32_t ba = saddr(s.kq[0][keys ? 0 : 1]), bk = saddr(s.kq[0][0]);
  float x[10][4];
  if (w & 1) pair_products<KP, true>(x, ba, bk, 2 * kTile, lane);
  else pair_products<KP, false>(x, ba, bk, 2 * kTile, lane);
  __syncthreads();   // K's and Q's memory is T's and P's from here
  // zeros above the diagonal: of rows r of 16, the units (of 8 columns) from 2 r + 2 on
  for (int i = tid; i < 4 * 64 * 6; i += kThreads) {
    const int row = i / 6 % 64, u = 2 + i % 6;
    if (u >= 2 * (row >> 4) + 2)
      *reinterpret_cast<uint4*>(s.tp[i / 384] + tile_at<64>(row, u)) = make_uint4(0, 0, 0, 0);
  }
  unsigned char* const to = keys ? s.a[0] : s.tp[2];
  if (s.vec[kSeg * kC + kC - 1] != 0.f) {
    if (w & 1) pair_decays<true, true>(x, s.vec, keys, a.scale, to, s.diag[0], lane);
    else pair_decays<false, true>(x, s.vec, keys, a.scale, to, s.diag[0], lane);
  } else {
    if (w & 1) pair_decays<true, false>(x, s.vec, keys, a.scale, to, s.diag[0], lane);
    else pair_decays<false, false>(x, s.vec, keys, a.scale, to, s.diag[0], lane);
  }
  __syncthreads();
  invert(s.tp[0], s.a[0], s.diag[0], w, lane, 1);
  tc::fence_proxy_async_smem();
  float* const vec = a.vec + id * vec_floats<kC>();
  for (int i = tid; i < kVecs * kC + 1; i += kThreads) vec[i] = s.vec[i];
  __syncthreads();
  if (tid == 0) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                     reinterpret_cast<unsigned char*>(a.T) + id * 4 * kTile),
                 "r"(saddr(s.tp[0])), "r"(4 * kTile)
                 : "memory");
    tc::bulk_commit();
    tc::bulk_wait_read();   // (the writes end with the kernel)
  }
}

template <int KP>
cudaError_t run(const Args& a, cudaStream_t st) {
  CUtensorMap mq, mk;
  if (!token_map(&mq, a.q, a.qcols, a.G, a.L, a.B, a.sq, true) ||
      !token_map(&mk, a.k, a.kcols, a.G, a.L, a.B, a.sk, true))
    return cudaErrorInvalidValue;
  const int smem = (int)sizeof(Smem<KP>) + 1024;
  const cudaError_t e = cudaFuncSetAttribute(
      tc_prepare_kernel<KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  g_launched = true;
  tc_prepare_kernel<KP><<<(unsigned)((int64_t)a.B * a.H * a.nc), kThreads, smem, st>>>(mq, mk, a);
  return cudaGetLastError();
}

}  // namespace prep

int tc_prepare_status(int reset, cudaStream_t st, int* bits) {
  return read_status(prep::g_status, prep::g_launched, reset, st, bits);
}
cudaError_t launch_tc_prepare(const Args& a, cudaStream_t st) {
  return a.KP == 64 ? prep::run<64>(a, st) : prep::run<128>(a, st);
}

}  // namespace delta
}  // namespace ssd
