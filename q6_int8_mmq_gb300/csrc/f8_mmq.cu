// Products of e4m3 blocks for many tokens:
//
//   Y[n][m] = sum_b sx[b][n] * sw[m / 128][b] * (sum_{k in b} xq[n][k] * wq[m][k])
//
// A pair of CTAs (cluster of two, cta_group::2) computes a tile of 256 tokens
// (MMA M; 128 tokens, one TMEM lane each, a CTA) by kBN weight rows. Each block
// of 128 of K is four tcgen05 MMAs (kind::f8f6f4, K = 32) into accumulators of
// its own, which eight warps of each CTA add, times the block's two scales, to
// f32 sums in registers while the next blocks' MMAs run: a thread has one token
// and columns of one block row of weights, so the product of the scales is one
// number a thread and block, and a value costs half a packed multiply-add.
//
// Warp roles (12 warps, persistent CTAs, one an SM): 0 loads tiles by TMA (128-
// byte swizzle), 1 of CTA 0 issues the pair's MMAs, 2 allocates TMEM, 4-11 sum:
// each warpgroup half of the tile's columns.
// TMEM: slots of kMmaN columns, 512 in all. A slot's MMAs are given out as soon
// as both CTAs have read what was in it.
// Every wait is bounded (see q6_internal.cuh), and the pair meets once more
// before either CTA leaves.
#include "f8_internal.cuh"
#include "f8_tc.cuh"

namespace q6 {
namespace {

constexpr int kThreads = 384;
constexpr int kTileN = 256;            // tokens of a pair
constexpr int kXTile = 128 * 128;      // bytes of a CTA's tokens of a stage
constexpr int kGroup = 8;              // token tiles walked together
// Registers of a thread: 128 + 256 threads share the 384 * 168 of the launch.
constexpr int kRegsFew = 72, kRegsMany = 216;

enum : uint32_t { kSiteEmpty = 48, kSiteFull, kSiteSlot, kSiteDone, kSiteDrain };

template <int kBN, int kMmaN>
struct Cfg {
  static constexpr int kUnits = kBN / kMmaN;      // accumulators of a block of K
  static constexpr int kSlots = 512 / kMmaN;
  static constexpr int kWRows = kBN / 2;          // of a CTA
  static constexpr int kStage = kXTile + kWRows * 128;
  static constexpr int kStages = kBN == 256 ? 6 : 8;
  static constexpr int kCols = kBN / 2;           // of a warpgroup
  // warps of the pair that read a slot
  static constexpr int kReaders = kUnits == 2 ? 8 : 16;
  struct Bars {
    uint64_t full[kStages], empty[kStages];
    uint64_t done[kSlots], taken[kSlots];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
  };
  static constexpr int kSmem = 1024 + kStages * kStage + (int)sizeof(Bars);
};

struct Maps {
  CUtensorMap x, w;
};

// D[tmem] (+)= A[smem] * B[smem]^T over the CTA pair, e4m3, f32 sums.
__device__ __forceinline__ void umma_f8_pair(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 ad, {%1, %5};\n\t"
      "mov.b64 bd, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], ad, bd, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kSw128DescHi)
      : "memory");
}
__device__ __forceinline__ void fma2(float2& acc, uint32_t a, uint32_t b, uint64_t s) {
  asm("{\n\t.reg .b64 v, c;\n\t"
      "mov.b64 v, {%2, %3};\n\t"
      "mov.b64 c, {%0, %1};\n\t"
      "fma.rn.f32x2 c, v, %4, c;\n\t"
      "mov.b64 {%0, %1}, c;\n\t}\n"
      : "+f"(acc.x), "+f"(acc.y)
      : "r"(a), "r"(b), "l"(s));
}

// Tile t: token tiles in groups of kGroup, a group's weight tiles one after
// another with its token tiles next to each other, so that what the pairs work on
// at a time shares both its tokens and its weights in L2.
struct Tile {
  int n, m;
};
__device__ __forceinline__ Tile tile_at(int t, int n_tiles, int m_tiles) {
  const int group = t / (kGroup * m_tiles), first = group * kGroup;
  const int here = min(kGroup, n_tiles - first), at = t - group * kGroup * m_tiles;
  return {first + at % here, at / here};
}

template <typename T, int kBN, int kMmaN>
__global__ void __launch_bounds__(kThreads, 1)
f8_mmq_kernel(const __grid_constant__ Maps maps, const F8Call c, unsigned int* status) {
  using S = Cfg<kBN, kMmaN>;
  constexpr int kStages = S::kStages, kSlots = S::kSlots, kUnits = S::kUnits;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  typename S::Bars* bars = reinterpret_cast<typename S::Bars*>(ring + kStages * S::kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), cluster = blockIdx.x / 2, clusters = gridDim.x / 2;
  volatile int* abort_flag = &bars->abort;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&bars->full[i], 1), mbar_init(&bars->empty[i], 1);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&bars->done[i], 1);
      mbar_init(&bars->taken[i], S::kReaders);  // used in CTA 0
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    mbar_fence_init();
    tma_prefetch_desc(&maps.x);
    tma_prefetch_desc(&maps.w);
  }
  if (warp == 2) tmem_alloc_pair(&bars->tmem_base, 512);
  griddep_wait();
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const int blocks = (c.K + kF8Block - 1) / kF8Block;
  const int m_tiles = (c.M + kBN - 1) / kBN, n_tiles = (c.N + kTileN - 1) / kTileN;
  const int tiles = m_tiles * n_tiles;
  bool ok = true;
  if (warp < 4) {
    regs_dealloc<kRegsFew>();
    if (warp == 0) {
      int g = 0;
      for (int t = cluster; t < tiles && ok; t += clusters) {
        const Tile w = tile_at(t, n_tiles, m_tiles);
        const int n0 = __shfl_sync(0xffffffffu, w.n * kTileN + 128 * rank, 0);
        const int m0 = __shfl_sync(0xffffffffu, w.m * kBN + kMmaN / 2 * rank, 0);
        for (int b = 0; b < blocks; ++b, ++g) {
          const int slot = g % kStages;
          if (!(ok = mbar_wait_warp(&bars->empty[slot], (g / kStages & 1) ^ 1, abort_flag, status,
                                    kSiteEmpty)))
            break;
          if (elect_one()) {
            uint8_t* at = ring + slot * S::kStage;
            if (rank == 0) mbar_arrive_expect_tx(&bars->full[slot], 2 * S::kStage);
            tma_load_2d_pair(at, &maps.x, &bars->full[slot], b * 128, n0);
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
              tma_load_2d_pair(at + kXTile + u * kMmaN / 2 * 128, &maps.w, &bars->full[slot], b * 128,
                               m0 + u * kMmaN);
          }
          __syncwarp();
        }
      }
      // the last stages' MMAs are through, and this CTA has been told, before it leaves
      for (int k = g > kStages ? g - kStages : 0; k < g && ok; ++k)
        ok = mbar_wait_warp(&bars->empty[k % kStages], k / kStages & 1, abort_flag, status, kSiteEmpty);
      if (!ok && lane == 0) {
        // Copies in flight land before the CTA exits. They count on a barrier of the
        // pair, so they are given 1 ms.
        for (const long long t0 = clock64(); clock64() - t0 < 2100000;) {
        }
      }
    } else if (warp == 1 && rank == 0) {
      const uint32_t base = sw128_desc_lo(smem_u32(ring));
      int g = 0, u = 0;
      for (int t = cluster; t < tiles && ok; t += clusters) {
        for (int b = 0; b < blocks && ok; ++b, ++g) {
          const int slot = g % kStages;
          if (!(ok = mbar_wait_warp(&bars->full[slot], g / kStages & 1, abort_flag, status, kSiteFull)))
            break;
#pragma unroll
          for (int h = 0; h < kUnits; ++h, ++u) {
            const int d = u % kSlots;
            if (!(ok = mbar_wait_warp(&bars->taken[d], (u / kSlots & 1) ^ 1, abort_flag, status,
                                      kSiteSlot)))
              break;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t x = base + slot * (S::kStage >> 4);
              const uint32_t w = x + ((kXTile + h * kMmaN / 2 * 128) >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_f8_pair(tmem + kMmaN * d, x + 2 * k, w + 2 * k, idesc_f8(256, kMmaN), k > 0);
              commit_pair(&bars->done[d]);
              if (h == kUnits - 1) commit_pair(&bars->empty[slot]);
            }
            __syncwarp();
          }
        }
      }
      if (elect_one()) {  // MMAs in flight end before TMEM is freed
        volatile int no_abort = 0;
        commit_own(&bars->drain);
        mbar_wait_bounded(&bars->drain, 0, &no_abort, status, kSiteDrain);
      }
      __syncwarp();
    }
  } else {
    regs_alloc<kRegsMany>();
    constexpr int kCols = S::kCols, kParts = kCols / 32;
    const int q = warp % 4, me = (warp - 4) / 4;
    // this warp's lanes and first column of a slot
    const uint32_t src = tmem + ((uint32_t)(32 * q) << 16) + (kUnits == 2 ? 0 : kCols * me);
    int u = kUnits == 2 ? me : 0;  // accumulators so far
    for (int t = cluster; t < tiles && ok; t += clusters) {
      const Tile w = tile_at(t, n_tiles, m_tiles);
      const int n = w.n * kTileN + 128 * rank + 32 * q + lane;
      const int m0 = w.m * kBN + kCols * me;
      const bool live = n < c.N;
      // past the last band of weights the last one again, whose result is not stored
      const float* sw = c.sw + (size_t)min(m0 / 128, (c.M - 1) / 128) * blocks;
      const float* sx = c.sx + n;
      float2 acc[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
      // scales two blocks ahead
      float x0 = live ? sx[0] : 0.0f, w0 = sw[0], x1 = 0.0f, w1 = 0.0f;
      if (blocks > 1) x1 = live ? sx[c.ldsx] : 0.0f, w1 = sw[1];
      for (int b = 0; b < blocks; ++b, u += kUnits) {
        const float sf = x0 * w0;
        uint64_t s;
        asm("mov.b64 %0, {%1, %1};" : "=l"(s) : "f"(sf));
        x0 = x1, w0 = w1;
        if (b + 2 < blocks) x1 = live ? sx[(size_t)(b + 2) * c.ldsx] : 0.0f, w1 = sw[b + 2];
        const int d = u % kSlots;
        if (!(ok = mbar_wait_warp(&bars->done[d], u / kSlots & 1, abort_flag, status, kSiteDone)))
          break;
        tc_fence_after();
        uint32_t v[2][32];
        tmem_ld32(src + kMmaN * d, v[0]);
        tmem_wait(v[0]);
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
          if (p + 1 < kParts) {
            tmem_ld32_before(src + kMmaN * d + 32 * (p + 1), v[(p + 1) & 1], v[p & 1]);
          } else {  // all is in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader_tmem(&bars->taken[d]);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i)
            fma2(acc[16 * p + i], v[p & 1][2 * i], v[p & 1][2 * i + 1], s);
          if (p + 1 < kParts) tmem_wait_ld_after(v[(p + 1) & 1], acc + 16 * p);
        }
      }
      if (ok && live) {
        T* y = static_cast<T*>(c.Y) + (size_t)n * c.ldy + m0;
        const int cols = c.M - m0;
        constexpr int kPer = 16 / sizeof(T);
        if (cols >= kCols && (reinterpret_cast<uintptr_t>(y) & 15) == 0) {
#pragma unroll
          for (int i = 0; i < kCols; i += kPer) {
            uint4 o;
            if constexpr (sizeof(T) == 4) {
              o.x = __float_as_uint(acc[i / 2].x), o.y = __float_as_uint(acc[i / 2].y);
              o.z = __float_as_uint(acc[i / 2 + 1].x), o.w = __float_as_uint(acc[i / 2 + 1].y);
            } else {
              o.x = pack2<T>(acc[i / 2].x, acc[i / 2].y);
              o.y = pack2<T>(acc[i / 2 + 1].x, acc[i / 2 + 1].y);
              o.z = pack2<T>(acc[i / 2 + 2].x, acc[i / 2 + 2].y);
              o.w = pack2<T>(acc[i / 2 + 3].x, acc[i / 2 + 3].y);
            }
            *reinterpret_cast<uint4*>(y + i) = o;
          }
        } else {
#pragma unroll
          for (int i = 0; i < kCols; ++i)
            if (i < cols) y[i] = from_f32<T>(i % 2 ? acc[i / 2].y : acc[i / 2].x);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <typename T, int kBN, int kMmaN>
cudaError_t launch_n(const Maps& maps, const F8Call& c, unsigned int* status, cudaStream_t s) {
  const long long tiles = (((long long)c.M + kBN - 1) / kBN) * (((long long)c.N + kTileN - 1) / kTileN);
  const unsigned pairs = (unsigned)(tiles < 76 ? tiles : 76);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<kBN, kMmaN>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, f8_mmq_kernel<T, kBN, kMmaN>, maps, c, status);
}
// Whether 128 weight rows a tile leave fewer rounds of half the work.
bool narrow(const F8Call& c) {
  const long long n = ((long long)c.N + kTileN - 1) / kTileN;
  const long long wide = n * (((long long)c.M + 255) / 256), thin = n * (((long long)c.M + 127) / 128);
  return (thin + 75) / 76 < 2 * ((wide + 75) / 76);
}
#ifndef F8_MMAN
#define F8_MMAN 128
#endif
template <typename T>
cudaError_t launch_t(const Maps& maps, const F8Call& c, bool thin, unsigned int* status,
                     cudaStream_t s) {
  return thin ? launch_n<T, 128, 128>(maps, c, status, s)
              : launch_n<T, 256, F8_MMAN>(maps, c, status, s);
}

}  // namespace

cudaError_t f8_tc_prepare() {
  cudaError_t e = cudaSuccess;
  auto raise = [&](auto kernel, int smem) {
    if (!e) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  };
  auto all = [&](auto t) {
    using T = decltype(t);
    raise(f8_mmq_kernel<T, 128, 128>, Cfg<128, 128>::kSmem);
    raise(f8_mmq_kernel<T, 256, F8_MMAN>, Cfg<256, F8_MMAN>::kSmem);
  };
  all(float());
  all(__nv_bfloat16());
  all(__half());
  return e;
}

int launch_f8_tc(const F8Call& c, cudaError_t* e, unsigned int* status, cudaStream_t s) {
  const bool thin = narrow(c);
  Maps maps;
  int rc;
  if ((rc = encode_f8_map(&maps.x, c.xq, c.N, c.K, 128, "xq")) ||
      (rc = encode_f8_map(&maps.w, c.wq, c.M, c.K, thin || F8_MMAN == 128 ? 64 : 128, "wq")))
    return rc;
  *e = c.type == Q6_TYPE_F32    ? launch_t<float>(maps, c, thin, status, s)
       : c.type == Q6_TYPE_BF16 ? launch_t<__nv_bfloat16>(maps, c, thin, status, s)
                                : launch_t<__half>(maps, c, thin, status, s);
  return Q6_OK;
}

}  // namespace q6
