// Low-rank adapters of many requests beside a shared projection:
//   out[n] = Y[n] + scale[a] * B[a] (A[a] x[n]),  a the adapter of token n.
// Tokens come grouped by adapter, so a tile of up to 16 or 32 tokens shares
// one A and one B.
//
// Two kernels. Shrink: T[i] = scale[a] A[a] x (K long, r wide), K split over
// the warps of a CTA and, when there are few tiles, over CTAs too; the parts
// are added in a fixed order. Expand: out = Y + B[a] T (r long, M wide).
//
// Both on warp-level tf32 MMAs. f16 and bf16 values are tf32 values as they
// are; an f32 factor (x, T) is split into a tf32 value and a tf32 remainder
// and multiplied twice (2^-21 of it is lost). The products are short next to
// the bytes: 2 r flops for each 4 to 8 bytes of X and Y.
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
template <typename TX, typename TW, int RT>
__global__ void __launch_bounds__(kThreads)
shrink_kernel(const LoraCall c) {
  constexpr int kRows = 16 * RT;
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

constexpr int kColsWarp = 32;  // columns a warp takes at a time

// out = Y + B T. Grid (tiles, column blocks of `cols`). JV: ranks a lane loads
// at a time (r is a multiple of 4 * JV). kVec: 16-byte rows of Y and out.
template <typename TW, int RT, int JV, bool kVec>
__global__ void __launch_bounds__(kThreads)
expand_kernel(const LoraCall c, int cols) {
  constexpr int kRows = 16 * RT;
  extern __shared__ float ts[];  // T of the tile: [kRows][r + 4]
  griddep_wait();
  const Tile tile = find_tile(c.offsets, c.L, kRows, blockIdx.x);
  if (tile.group < 0) return;
  const int m1 = min(c.M, ((int)blockIdx.y + 1) * cols);
  if (tile.group == c.L) {  // tokens without an adapter
    if (c.out == c.Y) return;
    for (int n = 0; n < tile.count; ++n) {
      const long long row = c.rows[tile.first + n];
      for (int m = (int)blockIdx.y * cols + threadIdx.x; m < m1; m += blockDim.x)
        c.out[row * c.ldo + m] = c.Y[row * c.ldy + m];
    }
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int ld = c.r + 4;
  for (int i = threadIdx.x; i < kRows * c.r; i += blockDim.x) {
    const int n = i / c.r, j = i % c.r;
    float v = 0.0f;
    if (n < tile.count)
      for (int s = 0; s < c.splits; ++s)
        v += c.part[((size_t)s * c.items + tile.first + n) * c.r + j];
    ts[n * ld + j] = v;
  }
  __syncthreads();
  long long row[RT][2];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = 16 * i + 8 * h + g;
      row[i][h] = n < tile.count ? c.rows[tile.first + n] : -1;
    }
  const TW* B = static_cast<const TW*>(c.B) + (size_t)tile.group * c.M * (size_t)c.r;
  for (int m0 = (int)blockIdx.y * cols + warp * kColsWarp; m0 < m1;
       m0 += (int)(blockDim.x / 32) * kColsWarp) {
    // column of this lane in MMA tile p: slots 2t, 2t + 1 of tiles 2q and
    // 2q + 1 are the four consecutive columns 16 q + 4 t..
    float acc[RT][4][4] = {};
    for (int j0 = 0; j0 < c.r; j0 += 4 * JV) {
      float w[4][JV];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int m = m0 + 16 * (p / 2) + 4 * (g / 2) + 2 * (p % 2) + g % 2;
        if (m < c.M) {
          load_16<TW, JV>(B + (size_t)m * c.r + j0 + JV * t, w[p]);
        } else {
#pragma unroll
          for (int q = 0; q < JV; ++q) w[p][q] = 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int q = 0; q < JV / 2; ++q) {
          const float2 f0 = *reinterpret_cast<const float2*>(ts + (16 * i + g) * ld + j0 + JV * t + 2 * q);
          const float2 f1 =
              *reinterpret_cast<const float2*>(ts + (16 * i + 8 + g) * ld + j0 + JV * t + 2 * q);
          const float v[4] = {f0.x, f1.x, f0.y, f1.y};
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float a, b;
            tf32_split(v[e], a, b);
            hi[e] = __float_as_uint(a);
            lo[e] = __float_as_uint(b);
          }
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const uint32_t b0 = __float_as_uint(w[p][2 * q]), b1 = __float_as_uint(w[p][2 * q + 1]);
            mma_tf32(acc[i][p], lo, b0, b1);
            mma_tf32(acc[i][p], hi, b0, b1);
          }
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (row[i][h] < 0) continue;
        const float* y = c.Y + row[i][h] * c.ldy;
        float* o = c.out + row[i][h] * c.ldo;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int m = m0 + 16 * q + 4 * t;
          const float v[4] = {acc[i][2 * q][2 * h], acc[i][2 * q][2 * h + 1],
                              acc[i][2 * q + 1][2 * h], acc[i][2 * q + 1][2 * h + 1]};
          if (kVec) {
            if (m < c.M) {
              const float4 a = *reinterpret_cast<const float4*>(y + m);
              *reinterpret_cast<float4*>(o + m) =
                  make_float4(a.x + v[0], a.y + v[1], a.z + v[2], a.w + v[3]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (m + e < c.M) o[m + e] = y[m + e] + v[e];
          }
        }
      }
  }
}

// The most tiles `items` items in L groups (and the section without one) can
// make.
long long most_tiles(long long items, int L, int rows) {
  const long long t = items / rows + L + 1;
  return t < items ? t : items;
}
int tile_rows(long long items, int L) {
  // 32-row tiles once the groups average more than 16 items
  return items > 16ll * L ? 32 : 16;
}

template <typename TX, typename TW>
cudaError_t shrink(const LoraCall& c, cudaStream_t s) {
  const int rows = tile_rows(c.items, c.L);
  const dim3 grid((unsigned)most_tiles(c.items, c.L, rows), (unsigned)c.splits,
                  (unsigned)((c.r + kRankBlock - 1) / kRankBlock));
  return launch_pdl(rows == 32 ? shrink_kernel<TX, TW, 2> : shrink_kernel<TX, TW, 1>, grid,
                    dim3(kThreads), 0, s, c);
}

template <typename TW, int RT, int JV>
cudaError_t expand_v(const LoraCall& c, bool vec, cudaStream_t s) {
  const long long tiles = most_tiles(c.items, c.L, 16 * RT);
  // column blocks: as wide as leaves about four CTAs an SM, so that T is
  // staged less often
  int cols = 1024;
  while (cols > 64 && tiles * ((c.M + cols - 1) / cols) < 4 * 152) cols /= 2;
  const dim3 grid((unsigned)tiles, (unsigned)((c.M + cols - 1) / cols));
  const int threads = cols >= 256 ? kThreads : cols;
  const size_t smem = (size_t)16 * RT * (c.r + 4) * 4;
  return launch_pdl(vec ? expand_kernel<TW, RT, JV, true> : expand_kernel<TW, RT, JV, false>, grid,
                    dim3(threads), smem, s, c, cols);
}
template <typename TW, int RT>
cudaError_t expand_r(const LoraCall& c, bool vec, cudaStream_t s) {
  return c.r % 32 == 0   ? expand_v<TW, RT, 8>(c, vec, s)
         : c.r % 16 == 0 ? expand_v<TW, RT, 4>(c, vec, s)
                         : expand_v<TW, RT, 2>(c, vec, s);
}

template <typename TW>
cudaError_t lora_t(const LoraCall& c, cudaStream_t s) {
  const cudaError_t e = c.xtype == Q6_TYPE_F32    ? shrink<float, TW>(c, s)
                        : c.xtype == Q6_TYPE_BF16 ? shrink<__nv_bfloat16, TW>(c, s)
                                                  : shrink<__half, TW>(c, s);
  if (e != cudaSuccess) return e;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(c.Y) | reinterpret_cast<uintptr_t>(c.out) |
                         (uintptr_t)(c.ldy * 4) | (uintptr_t)(c.ldo * 4) | (uintptr_t)(c.M * 4);
  return tile_rows(c.items, c.L) == 32 ? expand_r<TW, 2>(c, bits % 16 == 0, s)
                                       : expand_r<TW, 1>(c, bits % 16 == 0, s);
}

}  // namespace

int lora_splits(long long items, int L, int r, int K) {
  // K parts over CTAs until there are about two CTAs an SM, at least 256 of K
  // (one step a warp) each
  const int rows = tile_rows(items, L);
  const long long tiles = most_tiles(items, L, rows) * ((r + kRankBlock - 1) / kRankBlock);
  int splits = 1;
  while (splits < 16 && tiles * splits < 2 * 152 && (K / (2 * splits)) >= 256) splits *= 2;
  return splits;
}

cudaError_t launch_lora(const LoraCall& c, cudaStream_t s) {
  return c.type == Q6_TYPE_BF16 ? lora_t<__nv_bfloat16>(c, s) : lora_t<__half>(c, s);
}

}  // namespace q6
