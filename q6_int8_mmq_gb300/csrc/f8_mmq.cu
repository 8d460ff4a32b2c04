// Products of e4m3 blocks for many tokens:
//
//   Y[n][m] = sum_b sx[b][n] * sw[m / 128][b] * (sum_{k in b} xq[n][k] * wq[m][k])
//
// A pair of CTAs (cluster of two, cta_group::2) computes a tile of 256 tokens
// (MMA M; 128 tokens, one TMEM lane each, a CTA) by kBN weight rows (MMA N). Each
// block of 128 of K is four tcgen05 MMAs (kind::f8f6f4, 128 rows, K = 32), or eight,
// into an accumulator of its own, which eight warps of each CTA add, times the block's two scales, to
// f32 sums in registers while the next blocks' MMAs run: a thread has one token and
// columns of one block row of weights, so the product of the scales is one number a
// thread and block, and a value costs half a packed multiply-add.
//
// Warp roles (12 warps, persistent CTAs, one an SM):
//   0      loads tiles by TMA (128-byte swizzle)
//   1, 3   of CTA 0 issue the pair's MMAs, every other block each
//   2      allocates TMEM, loads the tokens' scales
//   4-11   sum: each warpgroup half of the tile's columns
// TMEM: slots of kBN columns, 512 in all. A block's MMAs wait for its stage of the
// ring to be full and for its slot to be taken by those who sum; `done` says that they
// are through, and so that the tokens' scales, counted with the stage's tiles, are there.
// 256 columns are taken and written in two halves, 64 columns of each warpgroup, so that
// MMAs go on while the second is read (3314 x 4096 x 11008: 109.6 -> 107.5 us).
// What bounds it is how fast sums are taken: a warp's block is a chain of a look at a
// barrier, loads from TMEM and a hand-back, about 450 cycles besides its multiply-
// adds, and from there to the next sums in the slot are 300 cycles of signals and 700
// of MMAs. So the scales bring no wait of their own: the tokens' come by the stage's
// barrier, the weights' in registers, 32 blocks at a time. (Measured on
// 8192 x 22016 x 4096, us: scales loaded by those who sum 716, waited for on a barrier of
// their own 682, multiplied by a warp of their own and this, both 531 to 567. That warp
// took 480 cycles a block, too long for 128 weight rows: 256 x 4096 x 4096 13.9 us, this
// 11.6. Sixteen warps that sum: 605 against 514. Slots of 128 columns for each warpgroup:
// 506, but 402 against 385 for 8192 x 8192 x 8192.)
// Where the tiles are few, clusters of two or four pairs split K (form_of()).
// Every wait is bounded (see q6_internal.cuh), and the cluster meets once
// more before any CTA leaves.
#include "f8_internal.cuh"
#include "f8_tc.cuh"

namespace q6 {
namespace {

constexpr int kThreads = 384;
constexpr int kTileN = 256;            // tokens of a pair
constexpr int kXTile = 128 * 128;      // bytes of a CTA's tokens of a stage

constexpr int kGroup = 8;              // token tiles walked together
constexpr int kScaleBytes = 128 * 4;   // a block's scales of a CTA's tokens
constexpr int kPart = 64;              // bytes of a row that are stored at a time
constexpr int kOutBytes = 32 * kPart;  // of a warp
// Registers of a thread: 128 + 256 threads share the 384 * 168 of the launch. (With 256
// weight rows the 16-bit forms spill 8 bytes, outside the loop over K's blocks: a product
// of 4864 x 4096 reads them back 17480 times with K = 1024 and with 4096.)
constexpr int kRegsFew = 40, kRegsMany = 232;

enum : uint32_t { kSiteDone = 48, kSiteFull, kSiteSlot, kSiteDrain };

template <int kBN>
struct Cfg {
  static constexpr int kSlots = 512 / kBN;
  static constexpr int kStage = kXTile + kBN / 2 * 128;  // bytes of a CTA
  // An even number: a barrier of a stage is then always waited for by the same of the two
  // warps that issue MMAs, phase by phase. (With an odd one, a warp whose blocks' copies
  // came early could be a whole ring ahead of the other and take the phase before the
  // last for the one that it waits for, which has the same parity.)
  static constexpr int kStages = kBN == 256 ? 4 : 6;
  static_assert(kStages % 2 == 0 && kSlots % 2 == 0);
  static constexpr int kCols = kBN / 2;           // of a warpgroup
  static constexpr int kHalves = kBN / 128;       // of a slot, taken one by one
  struct Bars {
    uint64_t full[kStages], done[kStages], taken[kSlots * kHalves];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
  };
  // Blocks whose tokens' scales are kept: a stage's MMAs are through only after all who
  // sum have read the slot kSlots blocks before, and so have added what came before that.
  static constexpr int kScales = kBN == 256 ? 8 : 16;
  static_assert(kScales > kStages + kSlots + 1);
  static constexpr int kSmem =
      1024 + kStages * kStage + 8 * 2 * kOutBytes + kScales * kScaleBytes + (int)sizeof(Bars);
};
constexpr int kReaders = 16;  // warps of the pair that read a slot

struct Maps {
  CUtensorMap x, w, sx, y;
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

// The address of CTA 0's `bar` from any CTA of the pair, and an arrival there as
// arrive_leader_tmem()'s.
__device__ __forceinline__ uint32_t leader_address(uint64_t* bar, uint32_t lead) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(bar)), "r"(lead));
  return a;
}
__device__ __forceinline__ void arrive_at_leader(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A box from shared memory to its place in global memory; what was begun since the
// last call as a group; and the wait until all but kLeft groups have been read.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tma_stores_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int kLeft>
__device__ __forceinline__ void tma_stores_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLeft) : "memory");
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

// Sixteen bytes of results: kPer of them from a thread's pairs of sums.
template <typename T>
__device__ __forceinline__ uint4 pack16(const float2* a) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(a[0].x), __float_as_uint(a[0].y), __float_as_uint(a[1].x),
                      __float_as_uint(a[1].y));
  else
    return make_uint4(pack2<T>(a[0].x, a[0].y), pack2<T>(a[1].x, a[1].y), pack2<T>(a[2].x, a[2].y),
                      pack2<T>(a[3].x, a[3].y));
}

// A part of 64 bytes of each of `rows` rows from shared memory to rows of Y that TMA does
// not take, `left` results of a row inside it: neighbouring lanes store neighbouring
// words, or single 16-bit results where rows start on odd ones. (A lane's own row from
// registers, a result at a time: 4000 x 11007 x 4096 bf16 took 499 us instead of 177.)
template <typename W, typename T>
__device__ __forceinline__ void store_rows(T* y, long long ldy, const uint8_t* from, int lane, int rows,
                                           int left) {
  constexpr int kLanes = kPart / (int)sizeof(W) < 32 ? kPart / (int)sizeof(W) : 32;  // of a row
  constexpr int kTurns = kPart / (int)sizeof(W) / kLanes, kWide = (int)(sizeof(W) / sizeof(T));
  if constexpr (sizeof(W) >= sizeof(T)) {
    const int first = lane / kLanes, at = lane % kLanes;
    for (int r = first; r < rows; r += 32 / kLanes) {
#pragma unroll
      for (int i = 0; i < kTurns; ++i) {
        const int word = at + i * kLanes, byte = word * (int)sizeof(W), m = word * kWide;
        const W v = *reinterpret_cast<const W*>(from + r * kPart + ((byte >> 4 ^ (r >> 1 & 3)) << 4) +
                                                (byte & 15));
        T* to = y + r * ldy + m;
        if (m + kWide <= left) *reinterpret_cast<W*>(to) = v;
        else if (kWide == 2 && m < left) *reinterpret_cast<uint16_t*>(to) = (uint16_t)v;
      }
    }
  }
}

template <typename T, int kBN, int kParts>
__global__ void __launch_bounds__(kThreads, 1)
f8_mmq_kernel(const __grid_constant__ Maps maps, const F8Call c, int store, unsigned int* status) {
  using S = Cfg<kBN>;
  constexpr int kStages = S::kStages, kSlots = S::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* out_stage = ring + kStages * S::kStage;
  float* scales = reinterpret_cast<float*>(out_stage + 8 * 2 * kOutBytes);
  typename S::Bars* bars = reinterpret_cast<typename S::Bars*>(scales + S::kScales * 128);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cluster = blockIdx.x / (2 * kParts), clusters = gridDim.x / (2 * kParts);
  // of the cluster's pairs, and of the pair's CTAs
  const int pair = kParts > 1 ? (int)cluster_rank() / 2 : 0, rank = (int)cluster_rank() % 2;
  const uint32_t lead = 2 * pair;
  // this pair's blocks of K
  const int all_blocks = (c.K + kF8Block - 1) / kF8Block;
  const int first = all_blocks * pair / kParts, blocks = all_blocks * (pair + 1) / kParts - first;
  const int m_tiles = (c.M + kBN - 1) / kBN, n_tiles = (c.N + kTileN - 1) / kTileN;
  const int tiles = m_tiles * n_tiles;
  const Tile tile_0 = tile_at(cluster, n_tiles, m_tiles);
  auto tile_of = [&](int t) { return t == cluster ? tile_0 : tile_at(t, n_tiles, m_tiles); };
  volatile int* abort_flag = &bars->abort;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars->full[i], 1);  // used in CTA 0
      mbar_init(&bars->done[i], 1);
    }
    for (int i = 0; i < kSlots * S::kHalves; ++i) mbar_init(&bars->taken[i], kReaders);  // used in CTA 0
    mbar_init(&bars->drain, 2);
    bars->abort = 0;
    mbar_fence_init();
    tma_prefetch_desc(&maps.x);
    tma_prefetch_desc(&maps.w);
    tma_prefetch_desc(&maps.sx);
  }
  if (warp == 2) tmem_alloc_pair(&bars->tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's barriers are initialised
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tmem = bars->tmem_base;
  bool ok = true;
  if (warp < 4) {
    regs_dealloc<kRegsFew>();
    if (warp == 0) {
      // ---------------------------------------------------------------- tiles --
      // (A block's turn is to be shorter than its 256 or 512 cycles of MMAs: with 64-bit
      // counts and their remainders it took 500.)
      int stage = 0, phase = 1, blocks_in = 0;
      for (int t = cluster; t < tiles && ok; t += clusters) {
        const Tile w = tile_of(t);
        const int n0 = __shfl_sync(0xffffffffu, w.n * kTileN + 128 * rank, 0);
        const int m0 = __shfl_sync(0xffffffffu, w.m * kBN + kBN / 2 * rank, 0);
#pragma unroll 1
        for (int k = 128 * first; k < 128 * (first + blocks); k += 128) {
          uint8_t* at = ring + stage * S::kStage;
          uint64_t* full = &bars->full[stage];
          if (blocks_in >= kStages &&
              !(ok = mbar_wait_warp(&bars->done[stage], phase, abort_flag, status, kSiteDone)))
            break;
          if (elect_one()) {
            if (rank == 0) mbar_arrive_expect_tx(full, 2 * (S::kStage + kScaleBytes));
            tma_load_2d_pair(at, &maps.x, full, k, n0, lead);
            tma_load_2d_pair(at + kXTile, &maps.w, full, k, m0, lead);
          }
          __syncwarp();
          blocks_in = min(blocks_in + 1, kStages);
          if (++stage == kStages) stage = 0, phase ^= 1;
        }
      }
      // the last stages' MMAs are through, and this CTA has been told, before it leaves
      for (int i = 0; i < blocks_in && ok; ++i) {
        if (--stage < 0) stage = kStages - 1, phase ^= 1;
        ok = mbar_wait_warp(&bars->done[stage], phase ^ 1, abort_flag, status, kSiteDone);
      }
      if (!ok && lane == 0) {
        // Copies in flight land before the CTA exits. They count on a barrier of the
        // pair, so they are given 1 ms.
        for (const long long t0 = clock64(); clock64() - t0 < 2100000;) {
        }
      }
    } else if (warp == 2) {
      // --------------------------------------------------------------- scales --
      // (counted on the stage's barrier with its tiles)
      int stage = 0, phase = 1, at = 0, blocks_in = 0;
      for (int t = cluster; t < tiles && ok; t += clusters) {
        const int n0 =
            __shfl_sync(0xffffffffu, tile_of(t).n * kTileN + 128 * rank, 0);
#pragma unroll 1
        for (int b = 0; b < blocks; ++b) {
          if (blocks_in >= kStages &&
              !(ok = mbar_wait_warp(&bars->done[stage], phase, abort_flag, status, kSiteDone)))
            break;
          if (elect_one())
            tma_load_2d_pair(scales + at * 128, &maps.sx, &bars->full[stage], n0, first + b, lead);
          __syncwarp();
          blocks_in = min(blocks_in + 1, kStages);
          at = (at + 1) % S::kScales;
          if (++stage == kStages) stage = 0, phase ^= 1;
        }
      }
    } else if (rank == 0) {
      // ----------------------------------------------------------------- MMAs --
      const uint32_t base = sw128_desc_lo(smem_u32(ring));
      // Everything is worked out before the waits: from a slot's last hand-back to its
      // MMAs is part of what bounds the kernel.
      const int all = (tiles - cluster + clusters - 1) / clusters * blocks;
      int g = warp >> 1, stage = g, full_phase = 0, slot = g, taken_phase = 1;
      for (; g < all; g += 2) {
        const uint32_t x = base + stage * (S::kStage >> 4), w = x + (kXTile >> 4);
        const uint32_t d = tmem + kBN * slot;
        if (!(ok = mbar_wait_warp(&bars->full[stage], full_phase, abort_flag, status, kSiteFull))) break;
        // half h: 64 rows of each CTA's weights, from the (64 h)th on
#pragma unroll
        for (int h = 0; h < S::kHalves; ++h) {
          if (!(ok = mbar_wait_warp(&bars->taken[slot * S::kHalves + h], taken_phase, abort_flag, status,
                                    kSiteSlot)))
            break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_f8_pair(d + 128 * h, x + 2 * k, w + 512 * h + 2 * k, idesc_f8(256, 128), k > 0);
            if (h == S::kHalves - 1) commit_pair(&bars->done[stage], lead);
          }
          __syncwarp();
        }
        if (!ok) break;
        if ((stage += 2) >= kStages) stage -= kStages, full_phase ^= 1;
        if ((slot += 2) >= kSlots) slot -= kSlots, taken_phase ^= 1;
      }
      if (elect_one()) {  // MMAs in flight end before TMEM is freed
        volatile int no_abort = 0;
        commit_own(&bars->drain);
        mbar_wait_bounded(&bars->drain, 0, &no_abort, status, kSiteDrain);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------------- sums --
    regs_alloc<kRegsMany>();
    constexpr int kCols = S::kCols, kMine = kParts > 1 ? kCols / 2 : kCols;  // columns summed, stored
    const int q = warp % 4, me = (warp - 4) / 4;
    // this warp's lanes and first column of a slot
    const uint32_t src = tmem + ((uint32_t)(32 * q) << 16) + 64 * me;
    const float* mine = scales + 32 * q + lane;
    const uint32_t leader = leader_address(&bars->taken[0], lead);
    int stage = 0, phase = 0, get = 0;
    bool seen = false;  // this lane has seen the next block done
    // The weights' scales: lane i has block i's of 32, the next 32 are on their way. (Past
    // the last band of weights the last one again, whose result is not stored.)
    auto weight_scale = [&](int t, int b) {
      if (t >= tiles) return 0.0f;
      const int band = min((tile_of(t).m * kBN + kCols * me) / 128, (c.M - 1) / 128);
      return b + lane < blocks ? c.sw[(size_t)band * all_blocks + first + b + lane] : 0.0f;
    };
    float sw = 0.0f, sw_next = weight_scale(cluster, 0);
    for (int t = cluster; t < tiles; t += clusters) {
      float2 acc[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
#pragma unroll 1
      for (int i = 0; i < blocks; ++i) {
        if (i % 32 == 0) {
          sw = sw_next;
          sw_next = i + 32 < blocks ? weight_scale(t, i + 32) : weight_scale(t + clusters, 0);
        }
        const float of_weights = __shfl_sync(0xffffffffu, sw, i % 32);
        ok = __all_sync(0xffffffffu, seen) ||
             mbar_wait_warp(&bars->done[stage], phase, abort_flag, status, kSiteDone);
        if (!ok) break;
        tc_fence_after();
        const int turn = get % kSlots;
        const uint32_t at = src + kBN * turn;
        const float f = mine[get * 128] * of_weights;
        uint64_t s;  // the product of the scales, in both halves
        asm("mov.b64 %0, {%1, %1};" : "=l"(s) : "f"(f));
        get = (get + 1) % S::kScales;
        if (++stage == kStages) stage = 0, phase ^= 1;
        auto add = [&](float2* to, const uint32_t(&v)[32]) {
#pragma unroll
          for (int j = 0; j < 16; ++j) fma2(to[j], v[2 * j], v[2 * j + 1], s);
        };
        // No load is in flight from one iteration to the next: the compiler does not
        // know that its registers are not to be moved before the wait.
        uint32_t va[32], vb[32];
        tmem_ld(at, va);
        tmem_ld(at + 32, vb);
        tmem_wait_ld2(va, vb);
        if constexpr (kCols == 128) {
          tc_fence_before();  // the first half is in registers
          __syncwarp();
          if (lane == 0) arrive_at_leader(leader + 16 * turn);
          add(acc, va);
          tmem_ld_after(at + 128, va, acc);
          add(acc + 16, vb);
          tmem_ld_after(at + 160, vb, acc + 16);
          tmem_wait_ld2(va, vb);
        }
        // all is in registers
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at_leader(leader + 8 * (S::kHalves * turn + S::kHalves - 1));
        // (a look at a barrier takes 200 cycles, so it comes before the last adds)
        seen = mbar_test_wait(&bars->done[stage], phase);
        add(acc + kCols / 2 - 32, va);
        add(acc + kCols / 2 - 16, vb);
      }
      const Tile w = tile_of(t);
      const int n0 = w.n * kTileN + 128 * rank + 32 * q;
      int m0 = w.m * kBN + kCols * me;
      if constexpr (kParts > 1) {
        // Two pairs add up a half each of a warp's columns (of four pairs the first two those
        // of warpgroup 0, the others those of 1). The others' sums of it come into their
        // rings, which nothing uses any more: [pair that sent][warp][four columns][lane].
        const int owner = kParts == 4 ? 2 * me : 0;
        float4* in = reinterpret_cast<float4*>(ring) + (warp - 4) * (kMine / 4) * 32 + lane;
        constexpr int kFrom = 8 * (kMine / 4) * 32;
        static_assert((kParts - 1) * kFrom * 16 <= kStages * S::kStage);
        cluster_sync();
        if (n0 < c.N) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int p = owner + h;
            if (p == pair) continue;
#pragma unroll
            for (int j = 0; j < kMine / 4; ++j) {
              const float2* a = acc + h * kMine / 2 + 2 * j;
              store_at(in + (pair - (pair > p)) * kFrom + 32 * j, 2 * p + rank,
                       make_float4(a[0].x, a[0].y, a[1].x, a[1].y));
            }
          }
          if (pair == owner + 1) {
#pragma unroll
            for (int j = 0; j < kMine / 2; ++j) acc[j] = acc[kMine / 2 + j];
          }
        }
        cluster_sync();
        if (pair < owner || pair > owner + 1) continue;
        if (n0 < c.N) {
#pragma unroll
          for (int i = 0; i < kParts - 1; ++i) {
#pragma unroll
            for (int j = 0; j < kMine / 4; ++j) {
              const float4 v = in[i * kFrom + 32 * j];
              acc[2 * j].x += v.x, acc[2 * j].y += v.y;
              acc[2 * j + 1].x += v.z, acc[2 * j + 1].y += v.w;
            }
          }
        }
        m0 += kMine * (pair - owner);
      }
      if (!ok) break;
      constexpr int kPer = kPart / (int)sizeof(T);  // results of a row stored at a time
      if (n0 >= c.N || m0 >= c.M) continue;
      // 64 bytes of 32 rows at a time, the 16-byte units of a row as the 64-byte swizzle has
      // them, so that a lane's row goes to banks of its own
      uint8_t* buf = out_stage + (warp - 4) * 2 * kOutBytes;
#pragma unroll
      for (int p = 0; p < kMine / kPer; ++p) {
        uint8_t* to = buf + (p & 1) * kOutBytes;
        if (p >= 2) {  // what was in the buffer has been read
          if (store == 16 && lane == 0) tma_stores_read<1>();
          __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(to + lane * kPart + ((j ^ (lane >> 1 & 3)) * 16)) =
              pack16<T>(acc + p * kPer / 2 + j * (8 / (int)sizeof(T)));
        if (store == 16) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (m0 + p * kPer < c.M) tma_store_2d(&maps.y, to, m0 + p * kPer, n0);
            tma_stores_commit();  // a group a part, with nothing in it past the last column
          }
        } else {
          __syncwarp();
          const int rows = min(32, c.N - n0), m = m0 + p * kPer;
          T* y = static_cast<T*>(c.Y) + (size_t)n0 * c.ldy + m;
          if (store == 4) store_rows<uint32_t, T>(y, c.ldy, to, lane, rows, c.M - m);
          else store_rows<uint16_t, T>(y, c.ldy, to, lane, rows, c.M - m);
        }
      }
      if (store == 16 && lane == 0) tma_stores_read<0>();
      __syncwarp();
    }
  }
  if (kParts > 1 && warp < 4) cluster_sync(), cluster_sync();  // those of the sums' way
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

long long tiles_of(long long n, int size) { return (n + size - 1) / size; }
template <int kBN, int kParts>
void launch_of(cudaLaunchConfig_t* cfg, cudaLaunchAttribute (&attr)[2], unsigned clusters, cudaStream_t s) {
  *cfg = {};
  cfg->gridDim = dim3(2 * kParts * clusters);
  cfg->blockDim = dim3(kThreads);
  cfg->dynamicSmemBytes = Cfg<kBN>::kSmem;
  cfg->stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2 * kParts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 2;
}
template <typename T, int kBN, int kParts>
cudaError_t launch_n(const Maps& maps, const F8Call& c, int store, unsigned int* status,
                     cudaStream_t s) {
  const long long tiles = tiles_of(c.M, kBN) * tiles_of(c.N, kTileN);
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  launch_of<kBN, kParts>(&cfg, attr, (unsigned)(kParts > 1 || tiles < 76 ? tiles : 76), s);
  return cudaLaunchKernelEx(&cfg, f8_mmq_kernel<T, kBN, kParts>, maps, c, store, status);
}
// Clusters of one, two and four pairs that a device holds at a time (each SM one CTA, the
// SMs of a cluster near one another): 76, 36 and 15 of 152 SMs.
struct Room {
  int of_one = 0, of_two = 0, of_four = 0;
};
Room g_room[kMaxDevices];  // written once, under the lock that every call takes

struct Form {
  bool thin;  // 128 weight rows a tile, not 256
  int parts;  // of K, a pair each
};
// 128 weight rows a tile take 5/8 of the time of 256 (600 x 14336 x 4096, five rounds of
// tiles against three: 45.7 us both; 512 x 11008 x 4096, three against two: 28.8, 31.5;
// 1536 x 11008 x 4096, seven against four: 63.3, 60.4). Where they leave most pairs without
// a tile, K is split: a block of K takes a pair 0.2 to 0.26 us, the sums' way to the pairs
// that add them up 1 us (two pairs) or 1.8 (four). (us, 256 tokens. 1024 weight rows, four
// pairs against one: K = 2048 6.6, 6.4; 2560 6.9, 7.3; 8192 10.3, 17.9. 4096 rows, two
// against one: K = 2560 9.0, 8.5; 3584 10.1, 10.3; 8192 15.3, 18.8.)
Form form_of(int M, int K, int N, const Room& room) {
  const long long n = tiles_of(N, kTileN), wide = n * tiles_of(M, 256), thin = n * tiles_of(M, 128);
  const int blocks = f8_blocks(K);
  if (5 * ((thin + 75) / 76) >= 8 * ((wide + 75) / 76)) return {false, 1};
  return {true, blocks >= 18 && thin <= room.of_four ? 4 : blocks >= 28 && thin <= room.of_two ? 2 : 1};
}
template <typename T>
cudaError_t launch_t(const Maps& maps, const F8Call& c, Form f, int store, unsigned int* status,
                     cudaStream_t s) {
  return !f.thin        ? launch_n<T, 256, 1>(maps, c, store, status, s)
         : f.parts == 1 ? launch_n<T, 128, 1>(maps, c, store, status, s)
         : f.parts == 2 ? launch_n<T, 128, 2>(maps, c, store, status, s)
                        : launch_n<T, 128, 4>(maps, c, store, status, s);
}

}  // namespace

cudaError_t f8_tc_prepare() {
  cudaError_t e = cudaSuccess;
  auto raise = [&](auto kernel, int smem) {
    if (!e) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  };
  auto all = [&](auto t) {
    using T = decltype(t);
    raise(f8_mmq_kernel<T, 128, 1>, Cfg<128>::kSmem);
    raise(f8_mmq_kernel<T, 128, 2>, Cfg<128>::kSmem);
    raise(f8_mmq_kernel<T, 128, 4>, Cfg<128>::kSmem);
    raise(f8_mmq_kernel<T, 256, 1>, Cfg<256>::kSmem);
  };
  all(float());
  all(__nv_bfloat16());
  all(__half());
  int device = 0;
  if (!e) e = cudaGetDevice(&device);
  if (e) return e;
  auto room = [](auto kernel, const cudaLaunchConfig_t& cfg) {
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) cudaGetLastError(), n = 0;  // none
    return n;
  };
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  launch_of<128, 1>(&cfg, attr, 1, nullptr);
  g_room[device].of_one = room(f8_mmq_kernel<float, 128, 1>, cfg);
  launch_of<128, 2>(&cfg, attr, 1, nullptr);
  g_room[device].of_two = room(f8_mmq_kernel<float, 128, 2>, cfg);
  launch_of<128, 4>(&cfg, attr, 1, nullptr);
  g_room[device].of_four = room(f8_mmq_kernel<float, 128, 4>, cfg);
  return e;
}

cudaError_t f8_tc_form(int M, int K, int N, F8Form* form) {
  int device = 0;
  const cudaError_t e = cudaGetDevice(&device);
  const Room& room = g_room[device];
  const Form f = form_of(M, K, N, room);
  *form = {kTileN, f.thin ? 128 : 256, f.parts,
           f.parts == 1 ? room.of_one : f.parts == 2 ? room.of_two : room.of_four};
  return e;
}

int launch_f8_tc(const F8Call& c, cudaError_t* e, unsigned int* status, cudaStream_t s) {
  int device = 0;
  if ((*e = cudaGetDevice(&device))) return Q6_OK;  // (the caller reports *e)
  const Form form = form_of(c.M, c.K, c.N, g_room[device]);
  // results by TMA where their rows start on 16 bytes, else in words of 4 or 2 bytes
  const int size = c.type == Q6_TYPE_F32 ? 4 : 2;
  const uintptr_t where = reinterpret_cast<uintptr_t>(c.Y) | (uintptr_t)(c.ldy * size);
  const int store = where % 16 == 0 ? 16 : where % 4 == 0 ? 4 : 2;
  Maps maps;
  int rc;
  if ((rc = encode_f8_map(&maps.x, c.xq, c.N, c.K, 128, "xq")) ||
      (rc = encode_f8_map(&maps.w, c.wq, c.M, c.K, form.thin ? 64 : 128, "wq")) ||
      (rc = encode_f8_scales(&maps.sx, c.sx, c.ldsx, f8_blocks(c.K), 128, 1)) ||
      (store == 16 && (rc = encode_f8_results(&maps.y, c, kPart / size, 32))))
    return rc;
  *e = c.type == Q6_TYPE_F32    ? launch_t<float>(maps, c, form, store, status, s)
       : c.type == Q6_TYPE_BF16 ? launch_t<__nv_bfloat16>(maps, c, form, store, status, s)
                                : launch_t<__half>(maps, c, form, store, status, s);
  return Q6_OK;
}

}  // namespace q6
