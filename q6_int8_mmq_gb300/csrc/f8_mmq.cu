// Products of e4m3 blocks:
//
//   Y[n][m] = sum_b sx[b][n] * sw[m / 128][b] * (sum_{k in b} xq[n][k] * wq[m][k])
//
// A CTA computes 128 tokens (MMA M, one TMEM lane each) by 128 weight rows.
// Each block of 128 of K is four tcgen05 MMAs (kind::f8f6f4, K = 32) into an
// accumulator of its own; while the next block's run, four warps add the
// finished one, times its two scales, to f32 sums in registers: a thread has one
// token and the tile lies in one block row of weights, so the product of the
// scales is one number a thread and block.
#include "f8_internal.cuh"
#include "f8_tc.cuh"

namespace q6 {
namespace {

constexpr int kThreads = 256;
constexpr int kStages = 5, kTile = 128 * 128, kStage = 2 * kTile;
constexpr int kSlots = 4, kTmemCols = 512;

enum : uint32_t { kSiteEmpty = 48, kSiteFull, kSiteSlot, kSiteDone, kSiteDrain };

struct Bars {
  uint64_t full[kStages], empty[kStages];
  uint64_t done[kSlots], taken[kSlots];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
constexpr int kSmemBytes = 1024 + kStages * kStage + (int)sizeof(Bars);

struct Maps {
  CUtensorMap x, w;
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
f8_mmq_kernel(const __grid_constant__ Maps maps, const F8Call c, unsigned int* status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Bars* bars = reinterpret_cast<Bars*>(ring + kStages * kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars->abort;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&bars->full[i], 1), mbar_init(&bars->empty[i], 1);
    for (int i = 0; i < kSlots; ++i) mbar_init(&bars->done[i], 1), mbar_init(&bars->taken[i], 4);
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    mbar_fence_init();
    tma_prefetch_desc(&maps.x);
    tma_prefetch_desc(&maps.w);
  }
  if (warp == 2) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const int blocks = (c.K + kF8Block - 1) / kF8Block;
  const int bands = (c.M + 127) / 128;
  const int mb = blockIdx.x % bands, n0 = blockIdx.x / bands * 128;
  bool ok = true;
  if (warp == 0) {
    int g = 0;
    for (; g < blocks; ++g) {
      const int slot = g % kStages;
      if (!(ok = mbar_wait_warp(&bars->empty[slot], (g / kStages & 1) ^ 1, abort_flag, status,
                                kSiteEmpty)))
        break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&bars->full[slot], kStage);
        tma_load_2d(ring + slot * kStage, &maps.x, &bars->full[slot], g * 128, n0);
        tma_load_2d(ring + slot * kStage + kTile, &maps.w, &bars->full[slot], g * 128, mb * 128);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) {  // copies in flight land before the CTA exits
      volatile int no_abort = 0;
      for (int k = g > kStages ? g - kStages : 0; k < g; ++k)
        mbar_wait_bounded(&bars->full[k % kStages], k / kStages & 1, &no_abort, status, kSiteFull);
    }
  } else if (warp == 1) {
    const uint32_t base = sw128_desc_lo(smem_u32(ring));
    for (int g = 0; g < blocks; ++g) {
      const int slot = g % kStages, d = g % kSlots;
      if (!(ok = mbar_wait_warp(&bars->taken[d], (g / kSlots & 1) ^ 1, abort_flag, status,
                                kSiteSlot)) ||
          !(ok = mbar_wait_warp(&bars->full[slot], g / kStages & 1, abort_flag, status, kSiteFull)))
        break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t a = base + slot * (kStage >> 4), b = a + (kTile >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_f8(tmem + 128 * d, a + 2 * k, b + 2 * k, idesc_f8(128, 128), k > 0);
        umma_commit(&bars->empty[slot]);
        umma_commit(&bars->done[d]);
      }
      __syncwarp();
    }
    if (elect_one()) {  // MMAs in flight end before TMEM is freed
      volatile int no_abort = 0;
      umma_commit(&bars->drain);
      mbar_wait_bounded(&bars->drain, 0, &no_abort, status, kSiteDrain);
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int q = warp % 4, n = n0 + 32 * q + lane;
    const uint32_t src = tmem + ((uint32_t)(32 * q) << 16);
    float acc[128];
#pragma unroll
    for (int i = 0; i < 128; ++i) acc[i] = 0.0f;
    const float* sw = c.sw + (size_t)mb * blocks;
    const bool live = n < c.N;
    float next = live ? c.sx[n] * sw[0] : 0.0f;
    for (int g = 0; g < blocks; ++g) {
      const int d = g % kSlots;
      const float s = next;
      if (g + 1 < blocks && live) next = c.sx[(size_t)(g + 1) * c.ldsx + n] * sw[g + 1];
      if (!(ok = mbar_wait_warp(&bars->done[d], g / kSlots & 1, abort_flag, status, kSiteDone)))
        break;
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t u[32], v[32];
        tmem_ld32(src + 128 * d + 64 * h, u);
        tmem_ld32(src + 128 * d + 64 * h + 32, v);
        tmem_wait_ld2(u, v);
        if (h == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->taken[d]);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          acc[64 * h + i] = fmaf(__uint_as_float(u[i]), s, acc[64 * h + i]);
          acc[64 * h + 32 + i] = fmaf(__uint_as_float(v[i]), s, acc[64 * h + 32 + i]);
        }
      }
    }
    if (ok && live) {
      T* y = static_cast<T*>(c.Y) + (size_t)n * c.ldy + mb * 128;
      const int cols = min(128, c.M - mb * 128);
#pragma unroll
      for (int i = 0; i < 128; ++i)
        if (i < cols) y[i] = from_f32<T>(acc[i]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <typename T>
cudaError_t launch_t(const Maps& maps, const F8Call& c, unsigned int* status, cudaStream_t s) {
  const unsigned grid = (unsigned)((c.M + 127) / 128) * (unsigned)((c.N + 127) / 128);
  return launch_pdl(f8_mmq_kernel<T>, dim3(grid), dim3(kThreads), kSmemBytes, s, maps, c, status);
}

}  // namespace

cudaError_t f8_tc_prepare() {
  cudaError_t e = cudaSuccess;
  auto raise = [&](auto kernel) {
    if (!e) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  };
  raise(f8_mmq_kernel<float>);
  raise(f8_mmq_kernel<__nv_bfloat16>);
  raise(f8_mmq_kernel<__half>);
  return e;
}

int launch_f8_tc(const F8Call& c, cudaError_t* e, unsigned int* status, cudaStream_t s) {
  Maps maps;
  int rc;
  if ((rc = encode_f8_map(&maps.x, c.xq, c.N, c.K, 128, "xq")) ||
      (rc = encode_f8_map(&maps.w, c.wq, c.M, c.K, 128, "wq")))
    return rc;
  *e = c.type == Q6_TYPE_F32    ? launch_t<float>(maps, c, status, s)
       : c.type == Q6_TYPE_BF16 ? launch_t<__nv_bfloat16>(maps, c, status, s)
                                : launch_t<__half>(maps, c, status, s);
  return Q6_OK;
}

}  // namespace q6
