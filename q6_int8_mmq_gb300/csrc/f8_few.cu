// Products of e4m3 blocks for a few tokens (see f8_mmq.cu for the formula).
//
// What bounds it is the weight, read once. It is the tensor cores' A operand as
// it lies in memory (128 rows, a TMEM lane each, by 128 of K: one TMA box with
// the 128-byte swizzle), so no instruction is spent on a weight: the tokens are
// B, 16 to 128 of them (MMA N). Each block's accumulator is added to f32 sums in
// registers by four warps (eight for 128 tokens), thread = weight row, times sw[b] * sx[b][n] of each
// token n.
//
// K is split over the CTAs of a cluster so that about two CTAs an SM stream
// weights; they exchange their sums through distributed shared memory, and each
// adds up a part of the results, in the order of K.
#include "f8_internal.cuh"
#include "f8_tc.cuh"

namespace q6 {
namespace {

constexpr int kWTile = 128 * 128;
constexpr int kMaxSplit = 8;

enum : uint32_t { kSiteEmpty = 56, kSiteFull, kSiteSlot, kSiteDone, kSiteDrain };

template <int kN>
struct Few {
  static constexpr int kStages = kN == 16 ? 6 : kN == 32 ? 5 : kN == 64 ? 4 : 3;
  static constexpr int kSlots = kN == 128 ? 2 : 4;
  // warps that sum, and a warp's tokens: so many that two CTAs' registers fit an SM
  static constexpr int kWarps = kN == 128 ? 8 : 4, kCols = kN * 4 / kWarps;
  static constexpr int kThreads = 64 + 32 * kWarps;
  static constexpr int kXTile = kN * 128, kStage = kWTile + kXTile;
  static constexpr int kSx = kN * 4 < 128 ? 128 : kN * 4;  // a stage's token scales
  struct Bars {
    uint64_t full[kStages], empty[kStages];
    uint64_t done[kSlots], taken[kSlots];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
  };
  static constexpr int kSmem = 1024 + kStages * (kStage + kSx) + (int)sizeof(Bars);
};

struct Maps {
  CUtensorMap x, w, sx;
};

// A value of the same place in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ float load_from(const float* p, int rank) {
  float v;
  asm volatile(
      "{\n\t.reg .b32 ra;\n\t"
      "mapa.shared::cluster.u32 ra, %1, %2;\n\t"
      "ld.shared::cluster.f32 %0, [ra];\n\t}\n"
      : "=f"(v)
      : "r"(smem_u32(p)), "r"(rank)
      : "memory");
  return v;
}

template <typename T, int kN>
__global__ void __launch_bounds__(Few<kN>::kThreads, 2)
f8_few_kernel(const __grid_constant__ Maps maps, const F8Call c, int split, unsigned int* status) {
  using S = Few<kN>;
  constexpr int kStages = S::kStages, kSlots = S::kSlots, kThreads = S::kThreads, kCols = S::kCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* scales = ring + kStages * S::kStage;
  typename S::Bars* bars = reinterpret_cast<typename S::Bars*>(scales + kStages * S::kSx);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars->abort;
  const int rank = blockIdx.x % split, mb = blockIdx.x / split;
  const int blocks = (c.K + kF8Block - 1) / kF8Block;
  const int first = (int)((long long)blocks * rank / split);
  const int last = (int)((long long)blocks * (rank + 1) / split);
  if (warp == 0 && elect_one()) {
    for (int i = 0; i < kStages; ++i) mbar_init(&bars->full[i], 1), mbar_init(&bars->empty[i], S::kWarps);
    for (int i = 0; i < kSlots; ++i) mbar_init(&bars->done[i], 1), mbar_init(&bars->taken[i], S::kWarps);
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    mbar_fence_init();
    // the weights' first tiles on their way into L2, which keeps them true to memory
    // should the kernel before still write them
    for (int b = first; b < last && b < first + kStages; ++b) tma_prefetch_2d(&maps.w, b * 128, mb * 128);
    tma_prefetch_desc(&maps.x);
    tma_prefetch_desc(&maps.sx);
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, kSlots * kN);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const int n_blocks = last - first;
  bool ok = true;
  float acc[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) acc[i] = 0.0f;
  // this thread's weight row and first token, in the warps that sum
  const int row = 32 * (warp & 3) + lane, n0 = (warp - 2) / 4 * kCols;
  if (warp == 0) {
    int g = 0;
    for (; g < n_blocks; ++g) {
      const int slot = g % kStages;
      if (!(ok = mbar_wait_warp(&bars->empty[slot], (g / kStages & 1) ^ 1, abort_flag, status,
                                kSiteEmpty)))
        break;
      if (elect_one()) {
        uint8_t* at = ring + slot * S::kStage;
        mbar_arrive_expect_tx(&bars->full[slot], S::kStage + kN * 4);
        tma_load_2d(at, &maps.w, &bars->full[slot], (first + g) * 128, mb * 128);
        tma_load_2d(at + kWTile, &maps.x, &bars->full[slot], (first + g) * 128, 0);
        tma_load_2d(scales + slot * S::kSx, &maps.sx, &bars->full[slot], 0, first + g);
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
    for (int g = 0; g < n_blocks; ++g) {
      const int slot = g % kStages, d = g % kSlots;
      if (!(ok = mbar_wait_warp(&bars->taken[d], (g / kSlots & 1) ^ 1, abort_flag, status,
                                kSiteSlot)) ||
          !(ok = mbar_wait_warp(&bars->full[slot], g / kStages & 1, abort_flag, status, kSiteFull)))
        break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t a = base + slot * (S::kStage >> 4), b = a + (kWTile >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_f8(tmem + kN * d, a + 2 * k, b + 2 * k, idesc_f8(128, kN), k > 0);
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
  } else {
    constexpr int kPart = kCols < 32 ? kCols : 32;  // columns read at a time
    const uint32_t src = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + n0;
    const float* sw = c.sw + (size_t)mb * blocks + first;
    float next = n_blocks > 0 ? sw[0] : 0.0f;
    for (int g = 0; g < n_blocks; ++g) {
      const int slot = g % kStages, d = g % kSlots;
      const float s = next;
      if (g + 1 < n_blocks) next = sw[g + 1];
      // the copies' barrier makes the scales visible, the MMAs' the sums
      if (!(ok = mbar_wait_warp(&bars->full[slot], g / kStages & 1, abort_flag, status, kSiteFull)) ||
          !(ok = mbar_wait_warp(&bars->done[d], g / kSlots & 1, abort_flag, status, kSiteDone)))
        break;
      tc_fence_after();
      const float4* sx = reinterpret_cast<const float4*>(scales + slot * S::kSx) + n0 / 4;
#pragma unroll
      for (int h = 0; h < kCols / kPart; ++h) {
        uint32_t v[kPart];
        tmem_ld(src + kN * d + kPart * h, v);
        tmem_wait(v);
#pragma unroll
        for (int i = 0; i < kPart; i += 4) {
          const float4 t = sx[(kPart * h + i) / 4];
          float* a = acc + kPart * h + i;
          a[0] = fmaf(__uint_as_float(v[i]), t.x * s, a[0]);
          a[1] = fmaf(__uint_as_float(v[i + 1]), t.y * s, a[1]);
          a[2] = fmaf(__uint_as_float(v[i + 2]), t.z * s, a[2]);
          a[3] = fmaf(__uint_as_float(v[i + 3]), t.w * s, a[3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->taken[d]), mbar_arrive(&bars->empty[slot]);
    }
    const int m = mb * 128 + row;
    if (split == 1) {
      if (m < c.M) {
        T* y = static_cast<T*>(c.Y) + (size_t)n0 * c.ldy + m;
#pragma unroll
        for (int i = 0; i < kCols; ++i)
          if (n0 + i < c.N) y[(size_t)i * c.ldy] = from_f32<T>(acc[i]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kSlots * kN);
  }
  if (split > 1) {
    // Sums [n][row] over the ring, which nothing reads or writes any more (every
    // stage was waited for). The cluster's CTAs add up tokens and rows in turn.
    float* sums = reinterpret_cast<float*>(ring);
    if (warp >= 2) {
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (n0 + i < c.N) sums[(n0 + i) * 128 + row] = acc[i];
    }
    cluster_sync();
    const int total = c.N * 128;
    for (int e = rank * kThreads + threadIdx.x; e < total; e += split * kThreads) {
      float v = load_from(sums + e, 0);
      for (int r = 1; r < split; ++r) v += load_from(sums + e, r);
      const int m = mb * 128 + e % 128;
      if (m < c.M) static_cast<T*>(c.Y)[(size_t)(e / 128) * c.ldy + m] = from_f32<T>(v);
    }
    cluster_sync();
  }
}

template <typename T, int kN>
cudaError_t launch_n(const Maps& maps, const F8Call& c, int split, unsigned int* status,
                     cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((c.M + 127) / 128) * (unsigned)split);
  cfg.blockDim = dim3(Few<kN>::kThreads);
  cfg.dynamicSmemBytes = Few<kN>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, f8_few_kernel<T, kN>, maps, c, split, status);
}
template <typename T>
cudaError_t launch_t(const Maps& maps, const F8Call& c, int n, int split, unsigned int* status,
                     cudaStream_t s) {
  return n == 16   ? launch_n<T, 16>(maps, c, split, status, s)
         : n == 32 ? launch_n<T, 32>(maps, c, split, status, s)
         : n == 64 ? launch_n<T, 64>(maps, c, split, status, s)
                   : launch_n<T, 128>(maps, c, split, status, s);
}

// Parts of K: as many as leave all CTAs resident, two an SM.
int split_of(const F8Call& c) {
  const long long bands = ((long long)c.M + 127) / 128;
  const int blocks = f8_blocks(c.K);
  long long split = 304 / bands;
  if (split > kMaxSplit) split = kMaxSplit;
  if (split > blocks) split = blocks;
  return split < 1 ? 1 : (int)split;
}

}  // namespace

cudaError_t f8_few_prepare() {
  cudaError_t e = cudaSuccess;
  auto raise = [&](auto kernel, int smem) {
    if (!e) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  };
  auto all = [&](auto t) {
    using T = decltype(t);
    raise(f8_few_kernel<T, 16>, Few<16>::kSmem);
    raise(f8_few_kernel<T, 32>, Few<32>::kSmem);
    raise(f8_few_kernel<T, 64>, Few<64>::kSmem);
    raise(f8_few_kernel<T, 128>, Few<128>::kSmem);
  };
  all(float());
  all(__nv_bfloat16());
  all(__half());
  return e;
}

int launch_f8_few(const F8Call& c, cudaError_t* e, unsigned int* status, cudaStream_t s) {
  const int n = c.N <= 16 ? 16 : c.N <= 32 ? 32 : c.N <= 64 ? 64 : 128;
  Maps maps;
  int rc;
  if ((rc = encode_f8_map(&maps.x, c.xq, c.N, c.K, n, "xq")) ||
      (rc = encode_f8_map(&maps.w, c.wq, c.M, c.K, 128, "wq")) ||
      (rc = encode_f8_scales(&maps.sx, c.sx, c.ldsx, f8_blocks(c.K), n, 1)))
    return rc;
  const int split = split_of(c);
  *e = c.type == Q6_TYPE_F32    ? launch_t<float>(maps, c, n, split, status, s)
       : c.type == Q6_TYPE_BF16 ? launch_t<__nv_bfloat16>(maps, c, n, split, status, s)
                                : launch_t<__half>(maps, c, n, split, status, s);
  return Q6_OK;
}

}  // namespace q6
