// Low-rank adapters of many requests beside a shared projection:
//   out[n] = Y[n] + scale[a] * B[a] (A[a] x[n]),  a the adapter of token n.
// Tokens come grouped by adapter, so a tile of up to 16 or 32 tokens shares
// one A and one B.
//
// Two kernels. Shrink: T[i] = scale[a] A[a] x (K long, r wide). For few tokens
// an adapter a CTA takes up to 16 of them and splits K over its warps; for
// many it takes 64, x and A coming through shared memory in four stages. K is
// also split over CTAs while there are few tiles; the parts are added in a
// fixed order. Expand: out = Y + B[a] T (r long, M wide), B in blocks of
// columns through shared memory, Y loaded a block ahead.
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

// kCount consecutive values as f32.
template <int kCount>
__device__ __forceinline__ void load_f32(const float* p, float (&f)[kCount]) {
#pragma unroll
  for (int i = 0; i < kCount / 4; ++i) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p) + i);
    f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
  }
}
template <typename T, int kCount>
__device__ __forceinline__ void load_16(const T* p, float (&f)[kCount]) {
  uint32_t w[kCount / 2];
  if constexpr (kCount == 8) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (kCount == 4) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  }
#pragma unroll
  for (int i = 0; i < kCount / 2; ++i) {
    const float2 v = unpack2<T>(w[i]);
    f[2 * i] = v.x, f[2 * i + 1] = v.y;
  }
}
template <int kCount>
__device__ __forceinline__ void load_f32(const __nv_bfloat16* p, float (&f)[kCount]) {
  load_16(p, f);
}
template <int kCount>
__device__ __forceinline__ void load_f32(const __half* p, float (&f)[kCount]) {
  load_16(p, f);
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

// T: part [split][item][r]. Grid (tiles, K splits, rank blocks).
template <typename TX, typename TW>
__global__ void __launch_bounds__(kThreads)
shrink_kernel(const LoraCall c) {
  constexpr int RT = 1, kRows = 16 * RT;
  constexpr bool kSplit = sizeof(TX) == 4;
  __shared__ float red[kWarps / 2][kRows][kRankBlock + 4];
  griddep_wait();
  griddep_launch_dependents();
  const Tile tile = find_tile(c.offsets, c.L, kRows, blockIdx.x);
  if (tile.group < 0 || tile.group == c.L) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int j0 = blockIdx.z * kRankBlock, nj = min(kRankBlock, c.r - j0) / 8;
  const TX* x[RT][2];
  bool has[RT][2];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = 16 * i + 8 * h + g;
      has[i][h] = n < tile.count;
      const long long row = c.rows[tile.first + (has[i][h] ? n : 0)];
      x[i][h] = static_cast<const TX*>(c.X) + row * c.ldx;
    }
  const TW* A = static_cast<const TW*>(c.A) +
                ((size_t)tile.group * c.r + j0 + g) * (size_t)c.K;
  float acc[RT][kRankBlock / 8][4] = {};
  // K in steps of 32, dealt out to (split, warp) in turn
  for (int k0 = ((int)blockIdx.y * kWarps + warp) * 32; k0 < c.K;
       k0 += (int)gridDim.y * kWarps * 32) {
    const int k = k0 + 8 * t;
    float f[RT][2][8];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (has[i][h]) {
          load_f32<8>(x[i][h] + k, f[i][h]);
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) f[i][h][q] = 0.0f;
        }
      }
#pragma unroll
    for (int j = 0; j < kRankBlock / 8; ++j) {
      if (j >= nj) break;
      float w[8];
      load_16<TW, 8>(A + (size_t)j * 8 * c.K + k, w);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        float p[4] = {};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t b0 = __float_as_uint(w[2 * q]), b1 = __float_as_uint(w[2 * q + 1]);
          const float v[4] = {f[i][0][2 * q], f[i][1][2 * q], f[i][0][2 * q + 1],
                              f[i][1][2 * q + 1]};
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float a, b;
            tf32_split(v[e], a, b);
            hi[e] = __float_as_uint(kSplit ? a : v[e]);
            lo[e] = __float_as_uint(b);
          }
          mma_tf32(p, hi, b0, b1);
          if constexpr (kSplit) mma_tf32(p, lo, b0, b1);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] += p[e];
      }
    }
  }
  // the warps' parts, halved three times: warp w takes warp w + half's
  for (int half = kWarps / 2; half; half /= 2) {
    if (warp >= half && warp < 2 * half) {
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < kRankBlock / 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j < nj) red[warp - half][16 * i + g + 8 * (e / 2)][8 * j + 2 * t + e % 2] = acc[i][j][e];
    }
    __syncthreads();
    if (warp < half) {
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < kRankBlock / 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j < nj) acc[i][j][e] += red[warp][16 * i + g + 8 * (e / 2)][8 * j + 2 * t + e % 2];
    }
    __syncthreads();
  }
  if (warp == 0) {
    const float scale = c.scale[tile.group];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < kRankBlock / 8; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = 16 * i + 8 * h + g;
          if (j < nj && n < tile.count) {
            float* p = c.part + ((size_t)blockIdx.y * c.items + tile.first + n) * c.r + j0 + 8 * j +
                       2 * t;
            *reinterpret_cast<float2*>(p) =
                make_float2(scale * acc[i][j][2 * h], scale * acc[i][j][2 * h + 1]);
          }
        }
  }
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
    for (int step = 0; step < 2; ++step) {  // 32 of K: 8 consecutive ones a lane
      // MMA i of 16 of K takes values 4 i.. of the lane's 8: a[i][part] its A
      // operand, the rows' values as they are or their parts
      constexpr bool kRaw = __is_same(TX, TW), kThree = kSplit && !__is_same(TW, __half);
      uint4 xw[2];    // kRaw
      float f[2][8];  // otherwise
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = row0 + 8 * h + g;
        if constexpr (kSplit) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int u = (8 * step + 2 * t + q) ^ (row & 1);
            const float4 v = *reinterpret_cast<const float4*>(x + (row * kXUnits + u) * 16);
            f[h][4 * q] = v.x, f[h][4 * q + 1] = v.y, f[h][4 * q + 2] = v.z, f[h][4 * q + 3] = v.w;
          }
        } else {
          const uint8_t* p = x + (row * kXUnits + ((4 * step + t) ^ ((row & 1) * 4))) * 16;
          if constexpr (kRaw)
            xw[h] = *reinterpret_cast<const uint4*>(p);
          else
            shared_f32<TX, 8>(p, f[h]);
        }
      }
      uint32_t three[2][3][4];  // [MMA][part][register]
      if constexpr (kThree) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // row e % 2, the pair 2 i + e / 2
            uint32_t p[3];
            const int k = 2 * (2 * i + e / 2);
            bf16_split3(f[e % 2][k], f[e % 2][k + 1], p);
#pragma unroll
            for (int s = 0; s < 3; ++s) three[i][s][e] = p[s];
          }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j >= nj) break;
        const int row = rank0 + 8 * j + g;
        const uint8_t* wp = x + kXBytes + (row * 8 + ((4 * step + t) ^ ((row & 1) * 4))) * 16;
        float p[4] = {};
        if constexpr (kRaw || kThree) {
          const uint4 w = *reinterpret_cast<const uint4*>(wp);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t b0 = word4(w, 2 * i), b1 = word4(w, 2 * i + 1);
            if constexpr (kRaw) {
              const uint32_t a[4] = {word4(xw[0], 2 * i), word4(xw[1], 2 * i),
                                     word4(xw[0], 2 * i + 1), word4(xw[1], 2 * i + 1)};
              mma_16<TW>(p, a, b0, b1);
            } else {
#pragma unroll
              for (int s = 2; s >= 0; --s) mma_16<TW>(p, three[i][s], b0, b1);
            }
          }
        } else {
          float w[8];
          shared_f32<TW, 8>(wp, w);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t b0 = __float_as_uint(w[2 * q]), b1 = __float_as_uint(w[2 * q + 1]);
            const float v[4] = {f[0][2 * q], f[1][2 * q], f[0][2 * q + 1], f[1][2 * q + 1]};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float a, b;
              tf32_split(v[e], a, b);
              hi[e] = __float_as_uint(kSplit ? a : v[e]);
              lo[e] = __float_as_uint(b);
            }
            if constexpr (kSplit) mma_tf32(p, lo, b0, b1);
            mma_tf32(p, hi, b0, b1);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] += p[e];
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

// out = Y + B T. Grid (tiles of 16 * RW items, column parts); RW row warps
// times col_warps column warps. JV: ranks a lane loads at a time (r is a
// multiple of 4 * JV). kVec: 16-byte rows of Y and out.
template <typename TW, int RW, int JV, bool kVec>
__global__ void __launch_bounds__(kThreads, 2)
expand_kernel(const LoraCall c, int col_warps, int part_cols) {
  constexpr int kRows = 16 * RW;
  extern __shared__ uint4 expand_smem[];
  float* ts = reinterpret_cast<float*>(expand_smem);  // T of the tile: [kRows][r + 4]
  const int ld = c.r + 4, pitch = b_pitch(c.r), width = kColsWarp * col_warps;
  uint8_t* bs = reinterpret_cast<uint8_t*>(ts + kRows * ld);  // two blocks of `width` columns
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int m_begin = (int)blockIdx.y * part_cols, m_end = min(c.M, m_begin + part_cols);
  griddep_wait();
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
  const int rw = warp % RW, cw = warp / RW;
  const float* ys[2];
  float* os[2];
  bool has[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = 16 * rw + 8 * h + g;
    has[h] = n < tile.count;
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
    for (int j0 = 0; j0 < c.r && !none; j0 += 4 * JV) {
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
  const bool big = many(c.items, c.L);
  const dim3 grid((unsigned)most_tiles(c.items, c.L, big ? kBigRows : 16), (unsigned)c.splits,
                  (unsigned)((c.r + kRankBlock - 1) / kRankBlock));
  if (big)
    return launch_pdl(shrink_big_kernel<TX, TW>, grid, dim3(kThreads),
                      (size_t)kBigStages * kBigStageBytes<TX, TW>, s, c);
  return launch_pdl(shrink_kernel<TX, TW>, grid, dim3(kThreads), 0, s, c);
}

size_t expand_smem_bytes(int rows, int r, int col_warps) {
  return (size_t)rows * (r + 4) * 4 + (size_t)2 * kColsWarp * col_warps * b_pitch(r);
}
constexpr size_t kExpandSmem = 112 * 1024;  // two CTAs an SM where that is enough
constexpr int kExpandSmemMax = 227 * 1024;
static_assert(128 * (Q6_LORA_MAX_RANK + 4) * 4 + 2 * kColsWarp * b_pitch(Q6_LORA_MAX_RANK) <=
                  kExpandSmemMax, "128 items at the largest rank");

template <typename TW, int RW, int JV>
cudaError_t expand_v(const LoraCall& c, bool vec, cudaStream_t s) {
  const long long tiles = most_tiles(c.items, c.L, 16 * RW);
  int col_warps = kWarps / RW;
  while (col_warps > 1 && (expand_smem_bytes(16 * RW, c.r, col_warps) > kExpandSmem ||
                           kColsWarp * col_warps >= 2 * c.M))
    col_warps /= 2;
  // column parts: about four CTAs an SM (two run at a time), whole blocks each
  const int width = kColsWarp * col_warps, blocks = (c.M + width - 1) / width;
  long long parts = (4 * 152 + tiles - 1) / tiles;
  if (parts > blocks) parts = blocks;
  const int part_cols = (int)((blocks + parts - 1) / parts) * width;
  const dim3 grid((unsigned)tiles, (unsigned)((c.M + part_cols - 1) / part_cols));
  return launch_pdl(vec ? expand_kernel<TW, RW, JV, true> : expand_kernel<TW, RW, JV, false>, grid,
                    dim3(32 * RW * col_warps), expand_smem_bytes(16 * RW, c.r, col_warps), s, c,
                    col_warps, part_cols);
}
template <typename TW, int RW>
cudaError_t expand_r(const LoraCall& c, bool vec, cudaStream_t s) {
  return c.r % 16 == 0 ? expand_v<TW, RW, 4>(c, vec, s) : expand_v<TW, RW, 2>(c, vec, s);
}

template <typename TW, int RW>
cudaError_t prepare_expand() {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto* k) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kExpandSmemMax);
  };
  set(expand_kernel<TW, RW, 4, true>), set(expand_kernel<TW, RW, 4, false>);
  set(expand_kernel<TW, RW, 2, true>), set(expand_kernel<TW, RW, 2, false>);
  return e;
}
template <typename TW>
cudaError_t prepare_t() {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto* k, int bytes) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  set(shrink_big_kernel<float, TW>, kBigStages * kBigStageBytes<float, TW>);
  set(shrink_big_kernel<__nv_bfloat16, TW>, kBigStages * kBigStageBytes<__nv_bfloat16, TW>);
  set(shrink_big_kernel<__half, TW>, kBigStages * kBigStageBytes<__half, TW>);
  if (e == cudaSuccess) e = prepare_expand<TW, 1>();
  if (e == cudaSuccess) e = prepare_expand<TW, 2>();
  return e;
}

template <typename TW>
cudaError_t lora_t(const LoraCall& c, cudaStream_t s) {
  const cudaError_t e = c.xtype == Q6_TYPE_F32    ? shrink<float, TW>(c, s)
                        : c.xtype == Q6_TYPE_BF16 ? shrink<__nv_bfloat16, TW>(c, s)
                                                  : shrink<__half, TW>(c, s);
  if (e != cudaSuccess) return e;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(c.Y) | reinterpret_cast<uintptr_t>(c.out) |
                         (uintptr_t)(c.ldy * 4) | (uintptr_t)(c.ldo * 4) | (uintptr_t)(c.M * 4);
  return many(c.items, c.L) ? expand_r<TW, 2>(c, bits % 16 == 0, s)
                            : expand_r<TW, 1>(c, bits % 16 == 0, s);
}

}  // namespace

int lora_splits(long long items, int L, int r, int K) {
  // K parts over CTAs, at least 256 of K each, as many as run at a time (two
  // CTAs an SM)
  const long long tiles = most_tiles(items, L, many(items, L) ? kBigRows : 16) *
                          ((r + kRankBlock - 1) / kRankBlock);
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
