// Products of e4m3 blocks for a few tokens (see f8_mmq.cu for the formula).
//
// What bounds it is the weight, read once. It is the tensor cores' A operand as
// it lies in memory (128 rows, a TMEM lane each, by 128 of K: one TMA box with
// the 128-byte swizzle), so no instruction is spent on a weight: the tokens are
// B, 16 to 64 of them (MMA N). Each block's accumulator is added to f32 sums in
// registers by four warps, thread = weight row, times sw[b] * sx[b][n] of each
// token n.
//
// K is split over the CTAs of a cluster so that about two CTAs an SM stream
// weights. Each sends its sums to the CTAs of the cluster that add up a part of them
// each, in the order of K, through distributed shared memory. A stage of the ring is free
// once its MMAs are through, not only after the sums, for which the tokens' scales stay
// (64 tokens: 22016 x 8192 43.4 -> 39.7 us, 11008 x 4096 13.2 -> 12.8; one token 11.0, the
// same. Blocks loaded two at a time: 47.5. Each band of weights from a block of its own
// on: 22016 x 4096 with one token 19.3 against 20.4, 4096 x 4096 5.8 against 5.7.)
#include "f8_internal.cuh"
#include "f8_tc.cuh"

namespace q6 {
namespace {

constexpr int kThreads = 192;
constexpr int kWTile = 128 * 128;
constexpr int kMaxSplit = 8;

enum : uint32_t { kSiteEmpty = 56, kSiteFull, kSiteSlot, kSiteDone, kSiteDrain };

template <int kN>
struct Few {
  static constexpr int kStages = kN == 16 ? 5 : kN == 32 ? 4 : 3;
  static constexpr int kSlots = 4;
  static constexpr int kXTile = kN * 128, kStage = kWTile + kXTile;
  static constexpr int kSx = kN * 4 < 128 ? 128 : kN * 4;  // a block's token scales
  // Blocks whose scales are kept: a stage is loaded anew after its MMAs, and those wait
  // for the sums kSlots blocks before to be in registers, and so for the ones before that.
  static constexpr int kScales = kN == 64 ? 8 : 16;
  static_assert(kScales > kStages + kSlots);
  // the cluster's sums that this CTA adds up: [CTA][a part of the tokens' rows]
  static constexpr int kSums = (32 * kN + kMaxSplit * kMaxSplit) * 16;
  struct Bars {
    uint64_t full[kStages], empty[kStages];
    uint64_t done[kSlots], taken[kSlots];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
  };
  static constexpr int kSmem = 1024 + kStages * kStage + kScales * kSx + kSums + (int)sizeof(Bars);
};

struct Maps {
  CUtensorMap x, w, sx;
};

// Four results next to each other, `left` of them inside Y; `vec`: they may be stored
// at once.
template <typename T>
__device__ __forceinline__ void store4(T* y, const float4& v, int left, bool vec) {
  if (vec && left >= 4) {
    if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(y) = v;
    else *reinterpret_cast<uint2*>(y) = make_uint2(pack2<T>(v.x, v.y), pack2<T>(v.z, v.w));
  } else {
    if (left > 0) y[0] = from_f32<T>(v.x);
    if (left > 1) y[1] = from_f32<T>(v.y);
    if (left > 2) y[2] = from_f32<T>(v.z);
    if (left > 3) y[3] = from_f32<T>(v.w);
  }
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

template <typename T, int kN>
__global__ void __launch_bounds__(kThreads, 2)
f8_few_kernel(const __grid_constant__ Maps maps, const F8Call c, int split, unsigned int* status) {
  using S = Few<kN>;
  constexpr int kStages = S::kStages, kSlots = S::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* scales = ring + kStages * S::kStage;
  float* sums = reinterpret_cast<float*>(scales + S::kScales * S::kSx);
  typename S::Bars* bars = reinterpret_cast<typename S::Bars*>(sums + S::kSums / 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars->abort;
  const int rank = blockIdx.x % split, mb = blockIdx.x / split;
  const int blocks = (c.K + kF8Block - 1) / kF8Block;
  const int first = (int)((long long)blocks * rank / split);
  const int last = (int)((long long)blocks * (rank + 1) / split);
  if (warp == 0 && elect_one()) {
    for (int i = 0; i < kStages; ++i) mbar_init(&bars->full[i], 1), mbar_init(&bars->empty[i], 1);
    for (int i = 0; i < kSlots; ++i) mbar_init(&bars->done[i], 1), mbar_init(&bars->taken[i], 4);
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
  if (split > 1) cluster_arrive();  // this CTA's shared memory may be written to
  griddep_wait();
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const int n_blocks = last - first;
  bool ok = true;
  float acc[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) acc[i] = 0.0f;
  const int quarter = warp & 3;  // of the 128 rows, in the warps that sum
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
        tma_load_2d(scales + g % S::kScales * S::kSx, &maps.sx, &bars->full[slot], 0, first + g);
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
  } else {
    constexpr int kPart = kN < 32 ? kN : 32;  // columns read at a time
    const uint32_t src = tmem + ((uint32_t)(32 * quarter) << 16);
    const float* sw = c.sw + (size_t)mb * blocks + first;
    // lane l has the scales of the weights' blocks l, 32 + l, ..., 32 blocks ahead (a load
    // takes longer than a block)
    auto fetch = [&](int g) { return g + lane < n_blocks ? sw[g + lane] : 0.0f; };
    float sw_now = 0.0f, sw_next = fetch(0);
    for (int g = 0; g < n_blocks; ++g) {
      const int d = g % kSlots;
      if (g % 32 == 0) sw_now = sw_next, sw_next = fetch(g + 32);
      const float s = __shfl_sync(0xffffffffu, sw_now, g % 32);
      // (MMAs that are through have waited for the block's copies, its scales among them)
      if (!(ok = mbar_wait_warp(&bars->done[d], g / kSlots & 1, abort_flag, status, kSiteDone))) break;
      tc_fence_after();
      const float4* sx = reinterpret_cast<const float4*>(scales + g % S::kScales * S::kSx);
#pragma unroll
      for (int h = 0; h < kN / kPart; ++h) {
        uint32_t v[kPart];
        tmem_ld(src + kN * d + kPart * h, v);
        tmem_wait(v);
        if (h == kN / kPart - 1) {  // all is in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->taken[d]);
        }
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
    }
    const int row = 32 * quarter + lane;
    if (split > 1) {
      // [token][row], over the ring: every stage was waited for, so nothing is under way
      float* own = reinterpret_cast<float*>(ring) + row;
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (i < c.N) own[128 * i] = acc[i];
    } else if (mb * 128 + row < c.M) {
      T* y = static_cast<T*>(c.Y) + mb * 128 + row;
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (i < c.N) y[(size_t)i * c.ldy] = from_f32<T>(acc[i]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kSlots * kN);
  }
  if (split > 1) {
    // Fours of rows of a token: CTA r adds up those from r * part on.
    const int fours = 32 * c.N, part = (fours + split - 1) / split;
    float4* in = reinterpret_cast<float4*>(sums);
    cluster_wait();
    for (int e = threadIdx.x; e < fours; e += kThreads) {
      const int to = e / part;
      store_at(in + rank * part + e - to * part, to, reinterpret_cast<const float4*>(ring)[e]);
    }
    cluster_arrive();
    cluster_wait();
    const bool vec = (reinterpret_cast<uintptr_t>(c.Y) | (uintptr_t)(c.ldy * (long long)sizeof(T))) %
                         (4 * sizeof(T)) == 0;
    for (int i = threadIdx.x; i < part && rank * part + i < fours; i += kThreads) {
      float4 v = in[i];
#pragma unroll
      for (int r = 1; r < kMaxSplit; ++r) {
        if (r < split) {
          const float4 p = in[r * part + i];
          v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
        }
      }
      const int e = rank * part + i, m = mb * 128 + e % 32 * 4;
      store4(static_cast<T*>(c.Y) + (size_t)(e / 32) * c.ldy + m, v, c.M - m, vec);
    }
  }
}

template <typename T, int kN>
cudaError_t launch_n(const Maps& maps, const F8Call& c, int split, unsigned int* status,
                     cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((c.M + 127) / 128) * (unsigned)split);
  cfg.blockDim = dim3(kThreads);
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
                   : launch_n<T, 64>(maps, c, split, status, s);
}

// Clusters of 1 to kMaxSplit CTAs that a device runs at a time, two CTAs an SM (a cluster's
// SMs are near one another): 304, 152, 97, 74, 58, 46, 38 and 36 of 152 SMs.
struct Room {
  int of[kMaxSplit + 1] = {};
};
Room g_room[kMaxDevices];  // written once, under the lock that every call takes
// Asked about in place of f8_few_kernel, of which the query counts one CTA an SM, as of
// every kernel that allocates TMEM; the same in threads and shared memory.
__global__ void __launch_bounds__(kThreads, 2) room_kernel() {}

// Parts of K: as many as leave the clusters of all bands of weights resident. (One token,
// K = 4096, us: 36 bands in eight parts 6.4; 37 in eight 9.1, in seven 6.5; 39 in seven 9.5, in
// six 6.6; 47 in six 11.5, in five 7.6; 59 in five 12.5, in four 8.6; 75 in four 13.6, in three
// 10.1; 98 in three 16.0, in two 12.9.)
int split_of(int M, int K, const Room& room) {
  const long long bands = ((long long)M + 127) / 128;
  int split = f8_blocks(K) < kMaxSplit ? f8_blocks(K) : kMaxSplit;
  while (split > 1 && bands > room.of[split]) --split;
  return split;
}
int width_of(int N) { return N <= 16 ? 16 : N <= 32 ? 32 : 64; }

}  // namespace

cudaError_t f8_few_prepare() {
  cudaError_t e = cudaSuccess;
  auto raise = [&](auto kernel, int smem) {
    if (!e) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    // two CTAs an SM want all of its shared memory
    if (!e)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
  };
  auto all = [&](auto t) {
    using T = decltype(t);
    raise(f8_few_kernel<T, 16>, Few<16>::kSmem);
    raise(f8_few_kernel<T, 32>, Few<32>::kSmem);
    raise(f8_few_kernel<T, 64>, Few<64>::kSmem);
  };
  all(float());
  all(__nv_bfloat16());
  all(__half());
  raise(room_kernel, Few<64>::kSmem);
  int device = 0;
  if (!e) e = cudaGetDevice(&device);
  if (e) return e;
  for (int i = 1; i <= kMaxSplit; ++i) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)i);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Few<64>::kSmem;  // the most of the three; two CTAs an SM with each
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)i;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int& n = g_room[device].of[i];
    if (cudaOccupancyMaxActiveClusters(&n, room_kernel, &cfg)) cudaGetLastError(), n = 0;
  }
  return e;
}

cudaError_t f8_few_form(int M, int K, int N, F8Form* form) {
  int device = 0;
  const cudaError_t e = cudaGetDevice(&device);
  if (e) return e;
  const int split = split_of(M, K, g_room[device]);
  *form = {width_of(N), 128, split, g_room[device].of[split]};
  return e;
}

int launch_f8_few(const F8Call& c, cudaError_t* e, unsigned int* status, cudaStream_t s) {
  int device = 0;
  if ((*e = cudaGetDevice(&device))) return Q6_OK;  // (the caller reports *e)
  const int n = width_of(c.N);
  Maps maps;
  int rc;
  if ((rc = encode_f8_map(&maps.x, c.xq, c.N, c.K, n, "xq")) ||
      (rc = encode_f8_map(&maps.w, c.wq, c.M, c.K, 128, "wq")) ||
      (rc = encode_f8_scales(&maps.sx, c.sx, c.ldsx, f8_blocks(c.K), n, 1)))
    return rc;
  const int split = split_of(c.M, c.K, g_room[device]);
  *e = c.type == Q6_TYPE_F32    ? launch_t<float>(maps, c, n, split, status, s)
       : c.type == Q6_TYPE_BF16 ? launch_t<__nv_bfloat16>(maps, c, n, split, status, s)
                                : launch_t<__half>(maps, c, n, split, status, s);
  return Q6_OK;
}

}  // namespace q6
