// Low-rank adapters of many requests beside a shared projection:
//   out[n] = Y[n] + scale[a] * B[a] (A[a] x[n]),  a the adapter of token n.
// Tokens come grouped by adapter, so a tile of up to 16 or 32 tokens shares
// one A and one B.
//
// Shrink: T[i] = scale[a] A[a] x (K long, r wide). Expand: out = Y + B[a] T (r
// long, M wide), B in blocks of columns through shared memory, Y loaded a block
// ahead. For few tokens an adapter one kernel does both: a CTA has up to 16
// tokens and a part of the columns, splits K over its 16 warps, and computes T
// again for each column part (A comes from L2 then; two kernels with K split
// over CTAs took 22 us for 47 tokens of 24 adapters of rank 32, 4096 x 11008).
// For many tokens an adapter there are two: shrink takes 64 tokens a CTA, x and
// A coming through shared memory in four stages, K split over CTAs and the parts
// added in a fixed order by expand, which takes 32.
//
// Both on warp-level MMAs with f32 accumulation, the 16-bit factors as they
// are. An f32 factor (x, T) beside bf16 is split into three bf16 values, 8
// bits each and together exact; beside f16 (whose range is too small for the
// parts) into a tf32 value and a tf32 remainder, which loses 2^-21 of it.
//
// The order of k inside an MMA is free, so a lane takes consecutive k (or
// rank) values of its row in 16-byte loads and the MMAs use them two by two.
//
// Bound: memory (X, Y and out once; the adapters in use once from HBM and
// once a tile from L2).
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
// A pair of f32 values as three bf16 pairs that add up to it.
__device__ __forceinline__ void bf16_split3(float x, float y, uint32_t (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    p[i] = __byte_perm(a, b, 0x7632u);  // the upper halves
    x -= __uint_as_float(a & 0xFFFF0000u);
    y -= __uint_as_float(b & 0xFFFF0000u);
  }
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
  __device__ __forceinline__ void prepare() {
    if constexpr (kThree) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // row e % 2, the pair 2 i + e / 2
          uint32_t p[3];
          const int k = 2 * (2 * i + e / 2);
          bf16_split3(value(e % 2, k), value(e % 2, k + 1), p);
#pragma unroll
          for (int s = 0; s < 3; ++s) three[i][s][e] = p[s];
        }
    }
  }
  // acc += this times 8 rows of A: a's words are the same 8 of K of row g.
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
          tf32_split(v[e], x, y);
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

// Shrink for many tokens an adapter. Grid (tiles of 64 items, K splits, rank
// blocks); warp w: items 16 (w % 4).., ranks 32 (w / 4)... Stages of 64 of K:
// x [64][64], A [64 ranks][64]; the 16-byte units of a row are exchanged by
// the row's lowest bit so that two rows' fragment loads meet no bank twice.
constexpr int kBigRows = 64, kBigStages = 4;
template <typename TX, typename TW>
constexpr int kBigStageBytes = kBigRows * 64 * (int)sizeof(TX) + kRankBlock * 64 * (int)sizeof(TW);

template <typename TX, typename TW>
__global__ void __launch_bounds__(kThreads, 2)
shrink_big_kernel(const LoraCall c) {
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
      xp.prepare();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j >= nj) break;
        const int row = rank0 + 8 * j + g;
        const int u = (4 * step + t) ^ ((row & 1) * 4);
        xp.multiply(*reinterpret_cast<const uint4*>(x + kXBytes + (row * 8 + u) * 16), acc[j]);
      }
    }
  }
  cp_async_wait<0>();
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

constexpr int kColsWarp = 64;  // columns a warp takes at a time

// Bytes of a column of B in shared memory: four neighbouring columns' fragment
// loads (32 bytes each) fall on different banks.
__host__ __device__ constexpr int b_pitch(int r) { return 2 * r + (2 * r % 64 == 0 ? 32 : 0); }

constexpr int kFusedThreads = 512, kFusedWarps = kFusedThreads / 32;
constexpr int kFusedSum = (kFusedWarps / 2) * 16 * (kRankBlock + 4) * 4;  // bytes of its partial sums

// T of a tile of up to 16 items into ts [16][ld], by all warps of a CTA, K dealt
// out to them 32 at a time; red: kFusedSum bytes.
template <typename TX, typename TW>
__device__ __forceinline__ void shrink_tile(const LoraCall& c, const Tile& tile, float* ts, int ld,
                                            float* red) {
  constexpr int kLoads = (int)sizeof(TX) / 2, kLd = kRankBlock + 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const TX* x[2];
  bool has[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    has[h] = 8 * h + g < tile.count;
    x[h] = static_cast<const TX*>(c.X) + c.rows[tile.first + (has[h] ? 8 * h + g : 0)] * c.ldx + 8 * t;
  }
  const float scale = c.scale[tile.group];
  for (int j0 = 0; j0 < c.r; j0 += kRankBlock) {
    const int nj = min(kRankBlock, c.r - j0) / 8;
    const TW* A = static_cast<const TW*>(c.A) +
                  ((size_t)tile.group * c.r + j0 + g) * (size_t)c.K + 8 * t;
    float acc[kRankBlock / 8][4] = {};
    for (int k = warp * 32; k < c.K; k += kFusedWarps * 32) {
      XPart<TX, TW> xp;
      uint4 w[kRankBlock / 8];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < kLoads; ++q)
          xp.put(h, q, has[h] ? __ldg(reinterpret_cast<const uint4*>(x[h] + k) + q)
                              : make_uint4(0, 0, 0, 0));
#pragma unroll
      for (int j = 0; j < kRankBlock / 8; ++j)
        if (j < nj) w[j] = __ldg(reinterpret_cast<const uint4*>(A + (size_t)j * 8 * c.K + k));
      xp.prepare();
#pragma unroll
      for (int j = 0; j < kRankBlock / 8; ++j)
        if (j < nj) xp.multiply(w[j], acc[j]);
    }
    // the warps' parts, halved until one has them all
    for (int half = kFusedWarps / 2; half; half /= 2) {
#pragma unroll
      for (int j = 0; j < kRankBlock / 8; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float2* p = reinterpret_cast<float2*>(red + ((warp % half) * 16 + 8 * h + g) * kLd + 8 * j + 2 * t);
          if (j < nj && warp >= half && warp < 2 * half)
            *p = make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
        }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kRankBlock / 8; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2* p =
              reinterpret_cast<const float2*>(red + ((warp % half) * 16 + 8 * h + g) * kLd + 8 * j + 2 * t);
          if (j < nj && warp < half) acc[j][2 * h] += p->x, acc[j][2 * h + 1] += p->y;
        }
      __syncthreads();
    }
    if (warp == 0) {
#pragma unroll
      for (int j = 0; j < kRankBlock / 8; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (j < nj)
            *reinterpret_cast<float2*>(ts + (8 * h + g) * ld + j0 + 8 * j + 2 * t) =
                make_float2(scale * acc[j][2 * h], scale * acc[j][2 * h + 1]);
    }
  }
}

// out = Y + B T. Grid (tiles of 16 * RW items, column parts); RW row warps
// times col_warps column warps. JV: ranks a lane loads at a time (r is a
// multiple of 4 * JV). kVec: 16-byte rows of Y and out. With TX (a type of X,
// RW = 1) it makes T itself and has kFusedThreads threads; with void T comes
// from shrink's parts.
template <typename TX, typename TW, int RW, int JV, bool kVec>
__global__ void __launch_bounds__(__is_same(TX, void) ? kThreads : kFusedThreads,
                                  __is_same(TX, void) ? 2 : 1)
expand_kernel(const LoraCall c, int col_warps, int part_cols) {
  constexpr bool kFused = !__is_same(TX, void);
  static_assert(!kFused || RW == 1, "the fused kernel has tiles of 16 items");
  constexpr int kRows = 16 * RW;
  extern __shared__ uint4 expand_smem[];
  float* ts = reinterpret_cast<float*>(expand_smem);  // T of the tile: [kRows][r + 4]
  const int ld = c.r + 4, pitch = b_pitch(c.r), width = kColsWarp * col_warps;
  uint8_t* bs = reinterpret_cast<uint8_t*>(ts + kRows * ld);  // two blocks of `width` columns
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int m_begin = (int)blockIdx.y * part_cols, m_end = min(c.M, m_begin + part_cols);
  griddep_wait();
  if (kFused) griddep_launch_dependents();
  const Tile tile = find_tile(c.offsets, c.L, kRows, blockIdx.x);
  if (tile.group < 0) return;
  const bool none = tile.group == c.L;  // tokens without an adapter: Y alone
  if (none && c.out == c.Y) return;
  const TW* B = static_cast<const TW*>(c.B) + (size_t)tile.group * c.M * (size_t)c.r;
  const int units = c.r / 8;  // 16-byte units of a column
  auto load = [&](int m0, int buf) {
    const int n = none ? 0 : min(width, m_end - m0) * units;
    for (int i = threadIdx.x; i < n; i += blockDim.x)
      cp_async16(bs + buf * width * pitch + i / units * pitch + i % units * 16,
                 B + (size_t)m0 * c.r + (size_t)i * 8, true);
    cp_async_commit();
  };
  load(m_begin, 0);
  if constexpr (kFused) {
    if (!none)
      shrink_tile<TX, TW>(c, tile, ts, ld, reinterpret_cast<float*>(bs + 2 * width * pitch));
  } else {
    // T, four ranks at a time, the parts' loads in flight together
    for (int i = threadIdx.x; i < kRows * (c.r / 4); i += blockDim.x) {
      const int n = i / (c.r / 4), j = i % (c.r / 4) * 4;
      float4 v = make_float4(0, 0, 0, 0);
      if (n < tile.count && !none) {
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
      *reinterpret_cast<float4*>(ts + n * ld + j) = v;
    }
  }
  const int rw = warp % RW, cw = warp / RW;
  const float* ys[2];
  float* os[2];
  bool has[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = 16 * rw + 8 * h + g;
    has[h] = n < tile.count && cw < col_warps;
    const long long row = c.rows[tile.first + (has[h] ? n : 0)];
    ys[h] = c.Y + row * c.ldy;
    os[h] = c.out + row * c.ldo;
  }
  // MMA tile p's slots 2t, 2t + 1 with those of tile p + 1 are the four
  // consecutive columns 16 (p / 2) + 4 t..
  const int col0 = cw * kColsWarp + 4 * t;
  auto load_y = [&](int h, int m) {
    return kVec && has[h] && m < m_end ? __ldcs(reinterpret_cast<const float4*>(ys[h] + m))
                                       : make_float4(0, 0, 0, 0);
  };
  float4 y[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < 4; ++q) y[h][q] = load_y(h, m_begin + col0 + 16 * q);
  int buf = 0;
  for (int m0 = m_begin; m0 < m_end; m0 += width, buf ^= 1) {
    if (m0 + width < m_end) {
      load(m0 + width, buf ^ 1);
    } else {
      cp_async_commit();
    }
    const int m = m0 + col0;
    cp_async_wait<1>();
    __syncthreads();  // the block (and, before the first, T) is there
    float acc[8][4] = {};
    const uint8_t* b = bs + buf * width * pitch + cw * kColsWarp * pitch;
    for (int j0 = 0; j0 < c.r && !none && cw < col_warps; j0 += 4 * JV) {
      constexpr bool kThree = JV == 4 && !__is_same(TW, __half);
      uint32_t hi[JV / 2][4], lo[JV / 2][4], three[3][4];
      float v[JV / 2][4];  // T of rows g, g + 8, two ranks each
#pragma unroll
      for (int q = 0; q < JV / 2; ++q) {
        const float* p = ts + (16 * rw + g) * ld + j0 + JV * t + 2 * q;
        const float2 f0 = *reinterpret_cast<const float2*>(p);
        const float2 f1 = *reinterpret_cast<const float2*>(p + 8 * ld);
        v[q][0] = f0.x, v[q][1] = f1.x, v[q][2] = f0.y, v[q][3] = f1.y;
      }
      if constexpr (kThree) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // row e % 2, the pair e / 2
          uint32_t p[3];
          bf16_split3(v[e / 2][e % 2], v[e / 2][2 + e % 2], p);
#pragma unroll
          for (int s = 0; s < 3; ++s) three[s][e] = p[s];
        }
      } else {
#pragma unroll
        for (int q = 0; q < JV / 2; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x, r;
            tf32_split(v[q][e], x, r);
            hi[q][e] = __float_as_uint(x);
            lo[q][e] = __float_as_uint(r);
          }
      }
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        // columns past M hold what the buffer held: they are not stored
        const int col = 16 * (p / 2) + 4 * (g / 2) + 2 * (p % 2) + g % 2;
        const uint8_t* wp = b + col * pitch + (j0 + JV * t) * 2;
        if constexpr (kThree) {
          const uint2 w = *reinterpret_cast<const uint2*>(wp);
#pragma unroll
          for (int s = 2; s >= 0; --s) mma_16<TW>(acc[p], three[s], w.x, w.y);
        } else {
          float w[JV];
          shared_f32<TW, JV>(wp, w);
#pragma unroll
          for (int q = 0; q < JV / 2; ++q) {
            const uint32_t b0 = __float_as_uint(w[2 * q]), b1 = __float_as_uint(w[2 * q + 1]);
            mma_tf32(acc[p], lo[q], b0, b1);
            mma_tf32(acc[p], hi[q], b0, b1);
          }
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int at = m + 16 * q;
        const float v[4] = {acc[2 * q][2 * h], acc[2 * q][2 * h + 1], acc[2 * q + 1][2 * h],
                            acc[2 * q + 1][2 * h + 1]};
        if (kVec) {
          const float4 a = y[h][q];
          if (has[h] && at < m_end)
            __stcs(reinterpret_cast<float4*>(os[h] + at),
                   make_float4(a.x + v[0], a.y + v[1], a.z + v[2], a.w + v[3]));
          y[h][q] = load_y(h, at + width);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (has[h] && at + e < m_end) os[h][at + e] = ys[h][at + e] + v[e];
        }
      }
    __syncthreads();  // the block has been read
  }
  cp_async_wait<0>();
}

// The most tiles `items` items in L groups (and the section without one) can
// make.
long long most_tiles(long long items, int L, int rows) {
  const long long t = items / rows + L + 1;
  return t < items ? t : items;
}
// Many tokens an adapter: more than 16 on average.
bool many(long long items, int L) { return items > 16ll * L; }

template <typename TX, typename TW>
cudaError_t shrink(const LoraCall& c, cudaStream_t s) {
  const dim3 grid((unsigned)most_tiles(c.items, c.L, kBigRows), (unsigned)c.splits,
                  (unsigned)((c.r + kRankBlock - 1) / kRankBlock));
  return launch_pdl(shrink_big_kernel<TX, TW>, grid, dim3(kThreads),
                    (size_t)kBigStages * kBigStageBytes<TX, TW>, s, c);
}

size_t expand_smem_bytes(int rows, int r, int col_warps) {
  return (size_t)rows * (r + 4) * 4 + (size_t)2 * kColsWarp * col_warps * b_pitch(r);
}
constexpr size_t kExpandSmem = 112 * 1024;  // two CTAs an SM where that is enough
constexpr int kExpandSmemMax = 227 * 1024;
constexpr int kBigRw = 2;  // row warps of the expand kernel for many tokens
static_assert(16 * (Q6_LORA_MAX_RANK + 4) * 4 + 2 * kColsWarp * b_pitch(Q6_LORA_MAX_RANK) + kFusedSum <=
                  kExpandSmemMax, "16 items at the largest rank");
static_assert(16 * kBigRw * (Q6_LORA_MAX_RANK + 4) * 4 + 2 * kColsWarp * b_pitch(Q6_LORA_MAX_RANK) <=
                  kExpandSmemMax, "the largest rank");

// The expand kernel for many tokens (TX void) or the fused one.
template <typename TX, typename TW, int JV>
cudaError_t expand_v(const LoraCall& c, bool vec, cudaStream_t s) {
  constexpr bool kFused = !__is_same(TX, void);
  constexpr int RW = kFused ? 1 : kBigRw;
  const long long tiles = most_tiles(c.items, c.L, 16 * RW);
  const size_t extra = kFused ? kFusedSum : 0;
  // column parts: about four CTAs an SM (two run at a time), or one of the
  // fused kernel, which makes T again in each; then the widest block that is
  // not wider than a part and leaves room
  const int cols = (c.M + kColsWarp - 1) / kColsWarp;  // in warps' columns
  long long parts = kFused ? 152 / tiles : (4 * 152 + tiles - 1) / tiles;
  parts = parts < 1 ? 1 : parts > cols ? cols : parts;
  int col_warps = kFused ? kFusedWarps : kWarps / RW;
  while (col_warps > 1 &&
         (expand_smem_bytes(16 * RW, c.r, col_warps) + extra > (kFused ? kExpandSmemMax : kExpandSmem) ||
          col_warps >= 2 * ((cols + parts - 1) / parts)))
    col_warps /= 2;
  const int width = kColsWarp * col_warps, blocks = (c.M + width - 1) / width;
  if (parts > blocks) parts = blocks;
  const int part_cols = (int)((blocks + parts - 1) / parts) * width;
  const dim3 grid((unsigned)tiles, (unsigned)((c.M + part_cols - 1) / part_cols));
  return launch_pdl(vec ? expand_kernel<TX, TW, RW, JV, true> : expand_kernel<TX, TW, RW, JV, false>,
                    grid, dim3(kFused ? kFusedThreads : 32 * RW * col_warps),
                    expand_smem_bytes(16 * RW, c.r, col_warps) + extra, s, c, col_warps, part_cols);
}
template <typename TX, typename TW>
cudaError_t expand(const LoraCall& c, cudaStream_t s) {
  const uintptr_t bits = reinterpret_cast<uintptr_t>(c.Y) | reinterpret_cast<uintptr_t>(c.out) |
                         (uintptr_t)(c.ldy * 4) | (uintptr_t)(c.ldo * 4) | (uintptr_t)(c.M * 4);
  const bool vec = bits % 16 == 0;
  return c.r % 16 == 0 ? expand_v<TX, TW, 4>(c, vec, s) : expand_v<TX, TW, 2>(c, vec, s);
}

template <typename TX, typename TW>
cudaError_t prepare_expand() {
  constexpr int RW = __is_same(TX, void) ? kBigRw : 1;
  cudaError_t e = cudaSuccess;
  auto set = [&](auto* k) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kExpandSmemMax);
  };
  set(expand_kernel<TX, TW, RW, 4, true>), set(expand_kernel<TX, TW, RW, 4, false>);
  set(expand_kernel<TX, TW, RW, 2, true>), set(expand_kernel<TX, TW, RW, 2, false>);
  return e;
}
template <typename TX, typename TW>
cudaError_t prepare_x() {
  cudaError_t e = cudaFuncSetAttribute(shrink_big_kernel<TX, TW>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kBigStages * kBigStageBytes<TX, TW>);
  return e == cudaSuccess ? prepare_expand<TX, TW>() : e;
}
template <typename TW>
cudaError_t prepare_t() {
  cudaError_t e = prepare_expand<void, TW>();
  if (e == cudaSuccess) e = prepare_x<float, TW>();
  if (e == cudaSuccess) e = prepare_x<__nv_bfloat16, TW>();
  if (e == cudaSuccess) e = prepare_x<__half, TW>();
  return e;
}

template <typename TX, typename TW>
cudaError_t lora_x(const LoraCall& c, cudaStream_t s) {
  if (!many(c.items, c.L)) return expand<TX, TW>(c, s);
  const cudaError_t e = shrink<TX, TW>(c, s);
  return e == cudaSuccess ? expand<void, TW>(c, s) : e;
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
