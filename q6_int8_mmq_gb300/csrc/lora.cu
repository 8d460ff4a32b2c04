// Low-rank adapters of many requests beside a shared projection:
//   out[n] = Y[n] + scale[a] * B[a] (A[a] x[n]),  a the adapter of token n.
// Tokens come grouped by adapter, so a tile of tokens (up to 4 where there are few, else
// 64 for A and 32 for B) shares one A and one B.
//
// Shrink: T[i] = scale[a] A[a] x (K long, r wide). Expand: out = Y + B[a] T (r
// long, M wide).
//
// Up to 8 tokens an adapter on average, one kernel does both on FMAs: a cluster
// of CTAs has up to 4 tokens of one adapter, each CTA a part of the columns and
// a part of K, whose sums they exchange through distributed shared memory. An
// MMA's 16 rows would be empty but for those tokens, and the loads are what
// counts: for 47 tokens of 24 adapters of rank 32 at 4096 x 11008 (25 MB), two MMA
// kernels with T in memory took 22 us, one MMA kernel that made T in each CTA
// 23 us, the same on FMAs 20 us, and with the sums shared 12.7 us.
//
// Beyond that there are two kernels on warp-level MMAs: shrink takes 64 tokens a
// CTA, x and A coming through shared memory in four stages, K split over CTAs
// and the parts added in a fixed order by expand, which takes 32 tokens, T split
// once, and whose warps each walk columns of their own, B copied and Y loaded a
// block ahead (sharing B among the warps of a CTA, with a barrier per block, took
// 73 instead of 68 us for 3314 tokens, rank 64, 11008 columns). MMAs with f32
// accumulation, the 16-bit factors as they are; an f32 factor (x, T) beside
// bf16 is split into three bf16 values, 8 bits each and together exact; beside
// f16 (whose range is too small for the parts) into a tf32 value and a tf32
// remainder, which loses 2^-21 of it.
//
// The order of k inside an MMA is free, so a lane takes consecutive k (or
// rank) values of its row in 16-byte loads and the MMAs use them two by two.
//
// Bound: memory at the least (X, Y and out once; the adapters in use once from HBM
// and once a tile from L2); expand by the latencies of 16 warps an SM (its factors
// from shared memory, MMAs, DRAM 40 % busy). 3314 tokens of 6 adapters of rank 64 at
// 4096 x 11008, 330 MB: 85 us, 3.9 TB/s (87 without reading B and Y before T is
// there; 1000 f16 tokens of 8 of rank 64 at 4096 x 4096 24.7 and 27.2).
#include <cuda_bf16.h>

#include "moe_internal.cuh"

namespace q6 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRankBlock = 64;  // ranks a shrink CTA holds

__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D += A (16 x 16) * B (16 x 8), 16-bit operands of type T.
template <typename T>
__device__ __forceinline__ void mma_16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                       uint32_t b1) {
  if constexpr (__is_same(T, __half))
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// What is left of x beside `part` of its bits. kInf: 0 of an infinity, which the part
// holds, instead of NaN. (NaN of a NaN, whose part may be an infinity.)
template <bool kInf>
__device__ __forceinline__ float rest(float x, float part) {
  return kInf && x == part ? 0.0f : x - part;
}
// A pair of f32 values as three bf16 pairs that add up to it.
template <bool kInf>
__device__ __forceinline__ void bf16_split3(float x, float y, uint32_t (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    p[i] = __byte_perm(a, b, 0x7632u);  // the upper halves
    if (i == 2) break;
    const float ah = __uint_as_float(a & 0xFFFF0000u), bh = __uint_as_float(b & 0xFFFF0000u);
    x = rest<kInf>(x, ah);
    y = rest<kInf>(y, bh);
  }
}
// An f32 value as a tf32 one and what is left of it.
template <bool kInf>
__device__ __forceinline__ void tf32_split2(float x, float& hi, float& lo) {
  tf32_split(x, hi, lo);
  lo = rest<kInf>(x, hi);
}

// The tile-th tile of kRows items, counted group by group (G = the section of
// items without an adapter): its group (-1 past the end), first item and
// number of items. Called by whole warps.
struct Tile {
  int group;
  long long first;
  int count;
};
__device__ __forceinline__ Tile find_tile(const int32_t* offsets, int G, int rows, int tile) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int g0 = 0; g0 <= G; g0 += 32) {
    const int g = g0 + lane;
    const int lo = g <= G ? offsets[g] : 0, hi = g <= G ? offsets[g + 1] : 0;
    const int mine = (hi - lo + rows - 1) / rows;
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int total = __shfl_sync(0xffffffffu, x, 31);
    if (tile < before + total) {
      const int at = tile - before;  // the first lane with x > at holds it
      const int src = __ffs(__ballot_sync(0xffffffffu, x > at)) - 1;
      const int in = at - (__shfl_sync(0xffffffffu, x, src) - __shfl_sync(0xffffffffu, mine, src));
      const int l = __shfl_sync(0xffffffffu, lo, src), h = __shfl_sync(0xffffffffu, hi, src);
      return Tile{g0 + src, (long long)l + (long long)in * rows, min(rows, h - l - in * rows)};
    }
    before += total;
  }
  return Tile{-1, 0, 0};
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool copy) {
  // copy == false fills with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(copy ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
// kCount values of shared memory as f32.
template <typename T, int kCount>
__device__ __forceinline__ void shared_f32(const void* p, float (&f)[kCount]) {
  uint32_t w[kCount / 2];
  if constexpr (kCount == 8) {
    const uint4 v = *static_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (kCount == 4) {
    const uint2 v = *static_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *static_cast<const uint32_t*>(p);
  }
#pragma unroll
  for (int i = 0; i < kCount / 2; ++i) {
    const float2 v = unpack2<T>(w[i]);
    f[2 * i] = v.x, f[2 * i + 1] = v.y;
  }
}

// 32 of K of two rows of x (g and g + 8 of a 16-row tile), 8 consecutive values
// a lane, ready for the products with as many of A.
template <typename TX, typename TW>
struct XPart {
  static constexpr bool kRaw = __is_same(TX, TW);  // the 16-bit words as they are
  static constexpr bool kThree = sizeof(TX) == 4 && !__is_same(TW, __half);
  static constexpr int kWords = 2 * (int)sizeof(TX);
  uint32_t w[2][kWords];  // the rows' values
  uint32_t three[2][3][4];  // [MMA][part][register]

  __device__ __forceinline__ void put(int row, int i, const uint4& v) {
    w[row][4 * i] = v.x, w[row][4 * i + 1] = v.y, w[row][4 * i + 2] = v.z, w[row][4 * i + 3] = v.w;
  }
  // Value k (0..7) of a row.
  __device__ __forceinline__ float value(int row, int k) const {
    if constexpr (sizeof(TX) == 4) {
      return __uint_as_float(w[row][k]);
    } else {
      const float2 f = unpack2<TX>(w[row][k / 2]);
      return k % 2 ? f.y : f.x;
    }
  }
  template <bool kInf>
  __device__ __forceinline__ void prepare() {
    if constexpr (kThree) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // row e % 2, the pair 2 i + e / 2
          uint32_t p[3];
          const int k = 2 * (2 * i + e / 2);
          bf16_split3<kInf>(value(e % 2, k), value(e % 2, k + 1), p);
#pragma unroll
          for (int s = 0; s < 3; ++s) three[i][s][e] = p[s];
        }
    }
  }
  // acc += this times 8 rows of A: a's words are the same 8 of K of row g.
  template <bool kInf>
  __device__ __forceinline__ void multiply(const uint4& a, float (&acc)[4]) const {
    float p[4] = {};
    if constexpr (kRaw || kThree) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t b0 = word4(a, 2 * i), b1 = word4(a, 2 * i + 1);
        if constexpr (kRaw) {
          const uint32_t x[4] = {w[0][2 * i], w[1][2 * i], w[0][2 * i + 1], w[1][2 * i + 1]};
          mma_16<TW>(p, x, b0, b1);
        } else {
#pragma unroll
          for (int s = 2; s >= 0; --s) mma_16<TW>(p, three[i][s], b0, b1);
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 b = unpack2<TW>(word4(a, q));
        const float v[4] = {value(0, 2 * q), value(1, 2 * q), value(0, 2 * q + 1),
                            value(1, 2 * q + 1)};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x, y;
          tf32_split2<kInf>(v[e], x, y);
          hi[e] = __float_as_uint(sizeof(TX) == 4 ? x : v[e]);
          lo[e] = __float_as_uint(y);
        }
        if constexpr (sizeof(TX) == 4)
          mma_tf32(p, lo, __float_as_uint(b.x), __float_as_uint(b.y));
        mma_tf32(p, hi, __float_as_uint(b.x), __float_as_uint(b.y));
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += p[e];
  }
};

template <bool kChoice>
struct Choice {
  static constexpr bool value = kChoice;
};

// Shrink for many tokens an adapter. Grid (tiles of 64 items, K splits, rank
// blocks); warp w: items 16 (w % 4).., ranks 32 (w / 4)... Stages of 64 of K:
// x [64][64], A [64 ranks][64]; the 16-byte units of a row are exchanged by
// the row's lowest bit so that two rows' fragment loads meet no bank twice.
constexpr int kBigRows = 64, kBigStages = 4;
template <typename TX, typename TW>
constexpr int kBigStageBytes = kBigRows * 64 * (int)sizeof(TX) + kRankBlock * 64 * (int)sizeof(TW);

template <typename TX, typename TW>
__global__ void __launch_bounds__(kThreads, 2)
shrink_kernel(const LoraCall c) {
  constexpr bool kSplit = sizeof(TX) == 4;
  constexpr int kXUnits = 64 * (int)sizeof(TX) / 16, kXSwap = kSplit ? 1 : 4;
  constexpr int kXBytes = kBigRows * 64 * (int)sizeof(TX), kStage = kBigStageBytes<TX, TW>;
  extern __shared__ uint4 big_smem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(big_smem);
  griddep_wait();
  griddep_launch_dependents();
  const Tile tile = find_tile(c.offsets, c.L, kBigRows, blockIdx.x);
  if (tile.group < 0 || tile.group == c.L) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int j0 = blockIdx.z * kRankBlock, ranks = min(kRankBlock, c.r - j0);
  // this CTA's stages of 64 of K
  const int stages = (c.K + 63) / 64;
  const int s0 = (int)((long long)stages * blockIdx.y / gridDim.y);
  const int s1 = (int)((long long)stages * (blockIdx.y + 1) / gridDim.y);
  // what a thread copies: units (row, u) of x and of A; rows past the end
  // repeat the last
  constexpr int kXCopies = kBigRows * kXUnits / kThreads, kACopies = kRankBlock * 8 / kThreads;
  const TX* xsrc[kXCopies];
  const TW* asrc[kACopies];
#pragma unroll
  for (int i = 0; i < kXCopies; ++i) {
    const int row = (threadIdx.x + i * kThreads) / kXUnits, u = (threadIdx.x + i * kThreads) % kXUnits;
    xsrc[i] = static_cast<const TX*>(c.X) +
              c.rows[tile.first + min(row, tile.count - 1)] * c.ldx + u * (16 / (int)sizeof(TX));
  }
#pragma unroll
  for (int i = 0; i < kACopies; ++i) {
    const int row = (threadIdx.x + i * kThreads) / 8, u = (threadIdx.x + i * kThreads) % 8;
    asrc[i] = static_cast<const TW*>(c.A) +
              ((size_t)tile.group * c.r + j0 + min(row, ranks - 1)) * (size_t)c.K + u * 8;
  }
  auto load = [&](int s) {
    if (s < s1) {
      uint8_t* x = smem + (s - s0) % kBigStages * kStage;
#pragma unroll
      for (int i = 0; i < kXCopies; ++i) {
        const int row = (threadIdx.x + i * kThreads) / kXUnits;
        const int u = (threadIdx.x + i * kThreads) % kXUnits;
        const bool in = s * 64 + u * (16 / (int)sizeof(TX)) < c.K;
        cp_async16(x + (row * kXUnits + (u ^ ((row & 1) * kXSwap))) * 16,
                   in ? xsrc[i] + (size_t)s * 64 : xsrc[i], in);
      }
#pragma unroll
      for (int i = 0; i < kACopies; ++i) {
        const int row = (threadIdx.x + i * kThreads) / 8, u = (threadIdx.x + i * kThreads) % 8;
        const bool in = s * 64 + u * 8 < c.K;
        cp_async16(x + kXBytes + (row * 8 + (u ^ ((row & 1) * 4))) * 16,
                   in ? asrc[i] + (size_t)s * 64 : asrc[i], in);
      }
    }
    cp_async_commit();
  };
  const int row0 = 16 * (warp % 4), rank0 = 32 * (warp / 4);
  const int nj = min(4, (ranks - rank0 + 7) / 8);
  float acc[4][4] = {};
  auto walk = [&](auto inf) {
    constexpr bool kInf = decltype(inf)::value;
#pragma unroll
    for (int s = 0; s < kBigStages - 1; ++s) load(s0 + s);
    for (int s = s0; s < s1; ++s) {
      cp_async_wait<kBigStages - 2>();
      __syncthreads();  // stage s is there, stage s - 1 has been read
      load(s + kBigStages - 1);
      const uint8_t* x = smem + (s - s0) % kBigStages * kStage;
#pragma unroll
      for (int step = 0; step < 2; ++step) {  // 32 of K
        XPart<TX, TW> xp;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = row0 + 8 * h + g;
          if constexpr (kSplit) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int u = (8 * step + 2 * t + q) ^ (row & 1);
              xp.put(h, q, *reinterpret_cast<const uint4*>(x + (row * kXUnits + u) * 16));
            }
          } else {
            const int u = (4 * step + t) ^ ((row & 1) * 4);
            xp.put(h, 0, *reinterpret_cast<const uint4*>(x + (row * kXUnits + u) * 16));
          }
        }
        xp.template prepare<kInf>();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j >= nj) break;
          const int row = rank0 + 8 * j + g;
          const int u = (4 * step + t) ^ ((row & 1) * 4);
          xp.template multiply<kInf>(
              *reinterpret_cast<const uint4*>(x + kXBytes + (row * 8 + u) * 16), acc[j]);
        }
      }
    }
    cp_async_wait<0>();
  };
  walk(Choice<false>());
  // An infinite f32 x has made NaN: again with the splits that keep it. (Those alone:
  // 3314 f32 tokens of rank 64 96.3 us, so 94.4, without either 94.0.)
  if constexpr (kSplit) {
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) odd |= isnan(acc[j][e]);
    if (__syncthreads_or(odd)) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
      walk(Choice<true>());
    }
  }
  const float scale = c.scale[tile.group];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = row0 + 8 * h + g;
      if (j < nj && n < tile.count) {
        float* p = c.part + ((size_t)blockIdx.y * c.items + tile.first + n) * c.r + j0 + rank0 +
                   8 * j + 2 * t;
        *reinterpret_cast<float2*>(p) = make_float2(scale * acc[j][2 * h], scale * acc[j][2 * h + 1]);
      }
    }
}

constexpr int kFewThreads = 512, kFewWarps = kFewThreads / 32;
constexpr int kFewItems = 4;  // of a tile

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// *p of CTA `rank` of the cluster.
__device__ __forceinline__ float load_cluster(const float* p, uint32_t rank) {
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

// A tile of up to kTok items' sums over this warp's K for ranks 8 j + g, j < nj,
// on FMAs (an MMA's 16 rows would be empty but for one to four, and splitting f32
// values for it costs more than the products): lane (g, t) takes 8 consecutive of
// 32 values of K, kSteps times those loaded together. This is warp `warp` of the
// `warps` that share K; sum[tok][8 j + g] is its own.
template <typename TX, typename TW, int kTok, int kNj>
__device__ __forceinline__ void shrink_fma(const LoraCall& c, const Tile& tile, const TW* A, int nj,
                                           int warp, int warps, float* sum) {
  constexpr int kSteps = 8 / kNj / kTok > 1 ? 8 / kNj / kTok : 1;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const TX* x[kTok];
#pragma unroll
  for (int n = 0; n < kTok; ++n)
    x[n] = static_cast<const TX*>(c.X) + c.rows[tile.first + min(n, tile.count - 1)] * c.ldx + 8 * t;
  float acc[kTok][kNj] = {};
  for (int k0 = warp * 32 * kSteps; k0 < c.K; k0 += warps * 32 * kSteps) {
    uint4 xw[kSteps][kTok][sizeof(TX) / 2], w[kSteps][kNj];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const bool in = k0 + 32 * s < c.K;
#pragma unroll
      for (int j = 0; j < kNj; ++j)
        w[s][j] = j < nj && in
                      ? __ldg(reinterpret_cast<const uint4*>(A + (size_t)j * 8 * c.K + k0 + 32 * s))
                      : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int n = 0; n < kTok; ++n)
#pragma unroll
        for (int q = 0; q < (int)sizeof(TX) / 2; ++q)
          xw[s][n][q] = in ? __ldg(reinterpret_cast<const uint4*>(x[n] + k0 + 32 * s) + q)
                           : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      float f[kTok][8];
#pragma unroll
      for (int n = 0; n < kTok; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (sizeof(TX) == 4) {
            f[n][2 * i] = __uint_as_float(word4(xw[s][n][i / 2], 2 * i % 4));
            f[n][2 * i + 1] = __uint_as_float(word4(xw[s][n][i / 2], 2 * i % 4 + 1));
          } else {
            const float2 v = unpack2<TX>(word4(xw[s][n][0], i));
            f[n][2 * i] = v.x, f[n][2 * i + 1] = v.y;
          }
        }
#pragma unroll
      for (int j = 0; j < kNj; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 a = unpack2<TW>(word4(w[s][j], i));
#pragma unroll
          for (int n = 0; n < kTok; ++n)
            acc[n][j] = fmaf(a.y, f[n][2 * i + 1], fmaf(a.x, f[n][2 * i], acc[n][j]));
        }
    }
  }
#pragma unroll
  for (int n = 0; n < kTok; ++n)
#pragma unroll
    for (int j = 0; j < kNj; ++j) {
      float v = acc[n][j];
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      v += __shfl_xor_sync(0xffffffffu, v, 2);
      if (t == 0 && j < nj) sum[n * kRankBlock + 8 * j + g] = v;
    }
}
template <typename TX, typename TW, int kTok>
__device__ __forceinline__ void shrink_few(const LoraCall& c, const Tile& tile, const TW* A, int nj,
                                           int rank, int ranks, float* red) {
  const int warp = threadIdx.x >> 5, warps = ranks * kFewWarps;
  float* sum = red + warp * kTok * kRankBlock;
  if (nj <= 2)
    shrink_fma<TX, TW, kTok, 2>(c, tile, A, nj, rank * kFewWarps + warp, warps, sum);
  else if (nj <= 4)
    shrink_fma<TX, TW, kTok, 4>(c, tile, A, nj, rank * kFewWarps + warp, warps, sum);
  else
    shrink_fma<TX, TW, kTok, 8>(c, tile, A, nj, rank * kFewWarps + warp, warps, sum);
}

// Both products for tiles of up to kFewItems items. Grid (tiles, column parts),
// clusters of `ranks` column parts.
template <typename TX, typename TW>
__global__ void __launch_bounds__(kFewThreads, 1)
lora_few_kernel(const LoraCall c, int part_cols, int ranks) {
  __shared__ float red[kFewWarps * kFewItems * kRankBlock];
  __shared__ float mine[kFewItems * Q6_LORA_MAX_RANK];              // this CTA's sums [item][r]
  __shared__ __align__(16) float ts[kFewItems * Q6_LORA_MAX_RANK];  // T [item][r]
  griddep_wait();
  griddep_launch_dependents();
  const Tile tile = find_tile(c.offsets, c.L, kFewItems, blockIdx.x);
  if (tile.group < 0) return;
  const bool none = tile.group == c.L;  // tokens without an adapter: Y alone
  if (none && c.out == c.Y) return;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int tok = tile.count == 1 ? 1 : kFewItems, rank = (int)blockIdx.y % ranks;
  for (int j0 = 0; j0 < c.r && !none; j0 += kRankBlock) {
    const int nj = min(kRankBlock, c.r - j0) / 8;
    const TW* A = static_cast<const TW*>(c.A) +
                  ((size_t)tile.group * c.r + j0 + g) * (size_t)c.K + 8 * t;
    if (tok == 1)
      shrink_few<TX, TW, 1>(c, tile, A, nj, rank, ranks, red);
    else
      shrink_few<TX, TW, kFewItems>(c, tile, A, nj, rank, ranks, red);
    __syncthreads();
    for (int i = threadIdx.x; i < tok * 8 * nj; i += kFewThreads) {
      const int n = i / (8 * nj), j = i % (8 * nj);
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) v += red[(w * tok + n) * kRankBlock + j];
      mine[n * c.r + j0 + j] = v;
    }
    __syncthreads();
  }
  if (!none) {
    cluster_sync_all();  // all CTAs' sums are there
    for (int i = threadIdx.x; i < tok * c.r; i += kFewThreads) {
      float v = 0.0f;
      for (int k = 0; k < ranks; ++k) v += load_cluster(mine + i, (uint32_t)k);
      ts[i] = c.scale[tile.group] * v;
    }
    cluster_sync_all();  // and have been read (no CTA leaves before)
  }
  const float* ys[kFewItems];
  float* os[kFewItems];
#pragma unroll
  for (int n = 0; n < kFewItems; ++n) {
    const long long row = c.rows[tile.first + min(n, tile.count - 1)];
    ys[n] = c.Y + row * c.ldy;
    os[n] = c.out + row * c.ldo;
  }
  // kCols columns a thread, their rows of B against T, 32 ranks at a time
  constexpr int kCols = 2;
  const TW* B = static_cast<const TW*>(c.B) + (size_t)tile.group * c.M * (size_t)c.r;
  const int m1 = min(c.M, ((int)blockIdx.y + 1) * part_cols);
  for (int m0 = (int)blockIdx.y * part_cols + threadIdx.x; m0 < m1; m0 += kCols * kFewThreads) {
    float y[kCols][kFewItems], add[kCols][kFewItems] = {};
#pragma unroll
    for (int p = 0; p < kCols; ++p)
#pragma unroll
      for (int n = 0; n < kFewItems; ++n)
        y[p][n] = n < tile.count && m0 + p * kFewThreads < m1 ? ys[n][m0 + p * kFewThreads] : 0.0f;
    for (int j0 = 0; j0 < c.r && !none; j0 += 32) {
      uint4 w[kCols][4];
#pragma unroll
      for (int p = 0; p < kCols; ++p)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int m = m0 + p * kFewThreads;
          w[p][u] = j0 + 8 * u < c.r && m < m1
                        ? __ldg(reinterpret_cast<const uint4*>(B + (size_t)m * c.r + j0 + 8 * u))
                        : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (j0 + 8 * u >= c.r) break;
        float f[kCols][8];
#pragma unroll
        for (int p = 0; p < kCols; ++p)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 v = unpack2<TW>(word4(w[p][u], i));
            f[p][2 * i] = v.x, f[p][2 * i + 1] = v.y;
          }
#pragma unroll
        for (int n = 0; n < kFewItems; ++n) {
          if (n >= tok) break;
          const float4* q = reinterpret_cast<const float4*>(ts + n * c.r + j0 + 8 * u);
          const float4 a = q[0], b = q[1];
          const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
          for (int p = 0; p < kCols; ++p)
#pragma unroll
            for (int i = 0; i < 8; ++i) add[p][n] = fmaf(f[p][i], v[i], add[p][n]);
        }
      }
    }
#pragma unroll
    for (int p = 0; p < kCols; ++p)
#pragma unroll
      for (int n = 0; n < kFewItems; ++n)
        if (n < tile.count && m0 + p * kFewThreads < m1)
          os[n][m0 + p * kFewThreads] = y[p][n] + add[p][n];
  }
}

// Expand for many tokens. A tile is 32 items; a CTA's warps take 32 columns each
// of its part in turn.
constexpr int kExpandRows = 32, kColsWarp = 32;  // a thread a column: blockDim.x is the width
// Bytes of a column of B in shared memory: four neighbouring columns' fragment
// loads (32 bytes each) fall on different banks.
__host__ __device__ constexpr int b_pitch(int r) { return 2 * r + (2 * r % 64 == 0 ? 32 : 0); }
// T in shared memory as the MMAs' factors: three bf16 parts [3][32][r + 8], or a
// tf32 value and the remainder [2][32][r + 4].
template <typename TW>
constexpr bool kThreeParts = !__is_same(TW, __half);
template <typename TW>
__host__ __device__ constexpr int t_pitch(int r) { return kThreeParts<TW> ? 2 * (r + 8) : 4 * (r + 4); }
template <typename TW>
constexpr int expand_smem(int r, int warps) {
  return (kThreeParts<TW> ? 3 : 2) * kExpandRows * t_pitch<TW>(r) + 2 * kColsWarp * warps * b_pitch(r);
}
// Warps of a CTA: 8, or as many as leave room for two CTAs an SM; 4 of one where
// two do not fit (rank 256).
constexpr int kExpandSmem = 112 * 1024, kExpandSmemMax = 227 * 1024;
template <typename TW>
constexpr int expand_warps(int r) {
  for (int w = kWarps; w > 1; w /= 2)
    if (expand_smem<TW>(r, w) <= kExpandSmem) return w;
  return 4;
}
static_assert(expand_smem<__nv_bfloat16>(Q6_LORA_MAX_RANK, 4) <= kExpandSmemMax &&
                  expand_smem<__half>(Q6_LORA_MAX_RANK, 4) <= kExpandSmemMax, "the largest rank");

// Grid (tiles, column parts). JV: ranks a lane loads at a time (r is a multiple
// of 4 * JV). kVec: 16-byte rows of Y and out.
template <typename TW, int JV, bool kVec>
__global__ void __launch_bounds__(kThreads, 2)
expand_kernel(const LoraCall c, int part_cols) {
  constexpr bool kThree = kThreeParts<TW>;
  constexpr int kParts = kThree ? 3 : 2;
  extern __shared__ uint4 smem_raw[];
  uint8_t* ts = reinterpret_cast<uint8_t*>(smem_raw);
  const int ld = t_pitch<TW>(c.r), pitch = b_pitch(c.r), width = (int)blockDim.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  // this warp's two blocks of B
  uint8_t* bs = ts + kParts * kExpandRows * ld + warp * 2 * kColsWarp * pitch;
  const int m_end = min(c.M, ((int)blockIdx.y + 1) * part_cols);
  const int m_first = (int)blockIdx.y * part_cols + warp * kColsWarp;
  // The kernel before is shrink, all of whose CTAs have passed their own wait once
  // this one runs: everything but T is in memory, and T is waited for below.
  const Tile tile = find_tile(c.offsets, c.L, kExpandRows, blockIdx.x);
  const bool none = tile.group == c.L;  // tokens without an adapter: Y alone
  if (tile.group < 0 || (none && c.out == c.Y)) {
    griddep_wait();
    return;
  }
  const TW* B = static_cast<const TW*>(c.B) + (size_t)tile.group * c.M * (size_t)c.r;
  const int units = c.r / 8;  // 16-byte units of a column
  auto load_b = [&](int m0, int buf) {
    const int n = none || m0 >= m_end ? 0 : min(kColsWarp, m_end - m0) * units;
    for (int i = lane; i < n; i += 32)
      cp_async16(bs + buf * kColsWarp * pitch + i / units * pitch + i % units * 16,
                 B + (size_t)m0 * c.r + (size_t)i * 8, true);
    cp_async_commit();
  };
  load_b(m_first, 0);
  const float* ys[4];  // rows g, g + 8, g + 16, g + 24 of the tile
  float* os[4];
  bool has[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    has[h] = 8 * h + g < tile.count;
    const long long row = c.rows[tile.first + (has[h] ? 8 * h + g : 0)];
    ys[h] = c.Y + row * c.ldy;
    os[h] = c.out + row * c.ldo;
  }
  auto load_y = [&](int h, int m) {
    return kVec && has[h] && m < m_end ? __ldcs(reinterpret_cast<const float4*>(ys[h] + m))
                                       : make_float4(0, 0, 0, 0);
  };
  // MMA tile p's slots 2t, 2t + 1 with those of tile p + 1 are the four
  // consecutive columns 16 (p / 2) + 4 t..
  float4 y[4][2];
#pragma unroll
  for (int h = 0; h < 4; ++h)
#pragma unroll
    for (int q = 0; q < 2; ++q) y[h][q] = load_y(h, m_first + 4 * t + 16 * q);
  griddep_wait();
  // T, four ranks at a time, the parts' loads in flight together
  for (int i = threadIdx.x; i < kExpandRows * (c.r / 4) && !none; i += width) {
    const int n = i / (c.r / 4), j = i % (c.r / 4) * 4;
    float4 v = make_float4(0, 0, 0, 0);
    if (n < tile.count) {
      const float* p = c.part + (size_t)(tile.first + n) * c.r + j;
      const size_t step = (size_t)c.items * c.r;
      for (int s0 = 0; s0 < c.splits; s0 += 8) {
        float4 w[8];
#pragma unroll
        for (int s = 0; s < 8; ++s)
          w[s] = s0 + s < c.splits ? *reinterpret_cast<const float4*>(p + (s0 + s) * step)
                                   : make_float4(0, 0, 0, 0);
#pragma unroll
        for (int s = 0; s < 8; ++s) v.x += w[s].x, v.y += w[s].y, v.z += w[s].z, v.w += w[s].w;
      }
    }
    uint8_t* to = ts + n * ld;
    if constexpr (kThree) {
      uint32_t a[3], b[3];
      bf16_split3<true>(v.x, v.y, a);
      bf16_split3<true>(v.z, v.w, b);
#pragma unroll
      for (int s = 0; s < 3; ++s)
        *reinterpret_cast<uint2*>(to + s * kExpandRows * ld + 2 * j) = make_uint2(a[s], b[s]);
    } else {
      float4 hi, lo;
      tf32_split2<true>(v.x, hi.x, lo.x), tf32_split2<true>(v.y, hi.y, lo.y);
      tf32_split2<true>(v.z, hi.z, lo.z), tf32_split2<true>(v.w, hi.w, lo.w);
      *reinterpret_cast<float4*>(to + 4 * j) = hi;
      *reinterpret_cast<float4*>(to + kExpandRows * ld + 4 * j) = lo;
    }
  }
  __syncthreads();
  int buf = 0;
  for (int m0 = m_first; m0 < m_end; m0 += width, buf ^= 1) {
    cp_async_wait<0>();
    __syncwarp();  // all lanes' copies of the block are there, the other block has been read
    load_b(m0 + width, buf ^ 1);
    float acc[2][4][4] = {};
    const uint8_t* b = bs + buf * kColsWarp * pitch;
    for (int j0 = 0; j0 < c.r && !none; j0 += 4 * JV) {
      // columns past M hold what the buffer held: they are not stored
      auto col_at = [&](int p) {
        return b + (16 * (p / 2) + 4 * (g / 2) + 2 * (p % 2) + g % 2) * pitch + (j0 + JV * t) * 2;
      };
      if constexpr (kThree && JV == 4) {
        uint32_t a[2][3][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int s = 0; s < 3; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint2 v = *reinterpret_cast<const uint2*>(
                  ts + (s * kExpandRows + 16 * i + 8 * h + g) * ld + (j0 + 4 * t) * 2);
              a[i][s][h] = v.x, a[i][s][2 + h] = v.y;
            }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint2 w = *reinterpret_cast<const uint2*>(col_at(p));
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int s = 2; s >= 0; --s) mma_16<TW>(acc[i][p], a[i][s], w.x, w.y);
        }
      } else {
        // tf32: the parts as they are (bf16 ones are tf32 values too)
        uint32_t a[kParts][JV / 2][2][4];
#pragma unroll
        for (int s = 0; s < kParts; ++s)
#pragma unroll
          for (int q = 0; q < JV / 2; ++q)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint8_t* p = ts + (s * kExpandRows + 16 * i + 8 * h + g) * ld;
                const int j = j0 + JV * t + 2 * q;
                float2 v;
                if constexpr (kThree)
                  v = unpack2<__nv_bfloat16>(*reinterpret_cast<const uint32_t*>(p + 2 * j));
                else
                  v = *reinterpret_cast<const float2*>(p + 4 * j);
                a[s][q][i][h] = __float_as_uint(v.x), a[s][q][i][2 + h] = __float_as_uint(v.y);
              }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          float w[JV];
          shared_f32<TW, JV>(col_at(p), w);
#pragma unroll
          for (int q = 0; q < JV / 2; ++q)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int s = kParts - 1; s >= 0; --s)
                mma_tf32(acc[i][p], a[s][q][i], __float_as_uint(w[2 * q]),
                         __float_as_uint(w[2 * q + 1]));
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int at = m0 + 4 * t + 16 * q;
        const float(&lo)[4] = acc[h / 2][2 * q], (&hi)[4] = acc[h / 2][2 * q + 1];
        const int e = 2 * (h % 2);
        const float v[4] = {lo[e], lo[e + 1], hi[e], hi[e + 1]};
        if (kVec) {
          const float4 a = y[h][q];
          if (has[h] && at < m_end)
            __stcs(reinterpret_cast<float4*>(os[h] + at),
                   make_float4(a.x + v[0], a.y + v[1], a.z + v[2], a.w + v[3]));
          y[h][q] = load_y(h, at + width);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (has[h] && at + k < m_end) os[h][at + k] = ys[h][at + k] + v[k];
        }
      }
  }
  cp_async_wait<0>();
}

// The most tiles `items` items in L groups (and the section without one) can
// make.
long long most_tiles(long long items, int L, int rows) {
  const long long t = items / rows + L + 1;
  return t < items ? t : items;
}
// Many tokens an adapter: more than 8 on average.
bool many(long long items, int L) { return items > 8ll * L; }

template <typename TX, typename TW>
cudaError_t shrink(const LoraCall& c, cudaStream_t s) {
  const dim3 grid((unsigned)most_tiles(c.items, c.L, kBigRows), (unsigned)c.splits,
                  (unsigned)((c.r + kRankBlock - 1) / kRankBlock));
  return launch_pdl(shrink_kernel<TX, TW>, grid, dim3(kThreads),
                    (size_t)kBigStages * kBigStageBytes<TX, TW>, s, c);
}

template <typename TW, int JV>
cudaError_t expand_v(const LoraCall& c, bool vec, cudaStream_t s) {
  const long long tiles = most_tiles(c.items, c.L, kExpandRows);
  const int warps = expand_warps<TW>(c.r), width = kColsWarp * warps;
  // Column parts, whole blocks each: about two CTAs an SM, as run at a time, or twice
  // that where T, which each CTA makes its factors of anew, is small. (Two against four
  // an SM, us: 3314 tokens, 6 adapters, M 11008, bf16 of rank 64, 80.4 to 97.9 by how
  // they fall against 84.8 to 85.7; 512 tokens, 4, M 4096, rank 16 9.8 / 8.5; f16 of
  // rank 64, 1000, 8, M 4096 24.7 / 27.1; bf16 of rank 128, 2048, 1, M 4096 52.0 / 57.9.)
  const int blocks = (c.M + width - 1) / width;
  const int t_bytes = (kThreeParts<TW> ? 3 : 2) * kExpandRows * t_pitch<TW>(c.r);
  const int an_sm = t_bytes <= 16 * 1024 ? 4 : 2;
  long long parts = (an_sm * 152 + tiles - 1) / tiles;
  if (parts > blocks) parts = blocks;
  const int part_cols = (int)((blocks + parts - 1) / parts) * width;
  const dim3 grid((unsigned)tiles, (unsigned)((c.M + part_cols - 1) / part_cols));
  return launch_pdl(vec ? expand_kernel<TW, JV, true> : expand_kernel<TW, JV, false>, grid,
                    dim3(32 * warps), (size_t)expand_smem<TW>(c.r, warps), s, c, part_cols);
}
template <typename TW>
cudaError_t expand(const LoraCall& c, cudaStream_t s) {
  const uintptr_t bits = reinterpret_cast<uintptr_t>(c.Y) | reinterpret_cast<uintptr_t>(c.out) |
                         (uintptr_t)(c.ldy * 4) | (uintptr_t)(c.ldo * 4) | (uintptr_t)(c.M * 4);
  const bool vec = bits % 16 == 0;
  return c.r % 16 == 0 ? expand_v<TW, 4>(c, vec, s) : expand_v<TW, 2>(c, vec, s);
}

template <typename TX, typename TW>
cudaError_t few(const LoraCall& c, cudaStream_t s) {
  // column parts: one CTA an SM, at least 128 columns; clusters of up to 8
  const long long tiles = most_tiles(c.items, c.L, kFewItems);
  long long parts = 152 / tiles;
  if (parts > c.M / 128) parts = c.M / 128;
  int ranks = 1;
  while (ranks < 8 && 2 * ranks <= parts) ranks *= 2;
  parts = parts < 1 ? 1 : parts / ranks * ranks;
  const int cols = (int)((c.M + parts - 1) / parts + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tiles, (unsigned)parts);
  cfg.blockDim = dim3(kFewThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = (unsigned)ranks;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, lora_few_kernel<TX, TW>, c, cols, ranks);
}

template <typename TW>
cudaError_t prepare_t() {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto* k, int bytes) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  constexpr int kMost = kExpandSmemMax;
  set(expand_kernel<TW, 4, true>, kMost), set(expand_kernel<TW, 4, false>, kMost);
  set(expand_kernel<TW, 2, true>, kMost), set(expand_kernel<TW, 2, false>, kMost);
  set(shrink_kernel<float, TW>, kBigStages * kBigStageBytes<float, TW>);
  set(shrink_kernel<__nv_bfloat16, TW>, kBigStages * kBigStageBytes<__nv_bfloat16, TW>);
  set(shrink_kernel<__half, TW>, kBigStages * kBigStageBytes<__half, TW>);
  return e;
}

template <typename TX, typename TW>
cudaError_t lora_x(const LoraCall& c, cudaStream_t s) {
  if (!many(c.items, c.L)) return few<TX, TW>(c, s);
  const cudaError_t e = shrink<TX, TW>(c, s);
  return e == cudaSuccess ? expand<TW>(c, s) : e;
}
template <typename TW>
cudaError_t lora_t(const LoraCall& c, cudaStream_t s) {
  return c.xtype == Q6_TYPE_F32    ? lora_x<float, TW>(c, s)
         : c.xtype == Q6_TYPE_BF16 ? lora_x<__nv_bfloat16, TW>(c, s)
                                   : lora_x<__half, TW>(c, s);
}

}  // namespace

int lora_splits(long long items, int L, int r, int K) {
  if (!many(items, L)) return 0;
  // K parts over CTAs, at least 256 of K each, as many as run at a time (two
  // CTAs an SM)
  const long long tiles = most_tiles(items, L, kBigRows) * ((r + kRankBlock - 1) / kRankBlock);
  long long splits = 2 * 152 / tiles;
  if (splits > K / 256) splits = K / 256;
  return splits < 1 ? 1 : splits > 16 ? 16 : (int)splits;
}

cudaError_t lora_prepare() {
  const cudaError_t e = prepare_t<__nv_bfloat16>();
  return e == cudaSuccess ? prepare_t<__half>() : e;
}

cudaError_t launch_lora(const LoraCall& c, cudaStream_t s) {
  return c.type == Q6_TYPE_BF16 ? lora_t<__nv_bfloat16>(c, s) : lora_t<__half>(c, s);
}

}  // namespace q6
