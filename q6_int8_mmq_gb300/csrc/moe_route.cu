// Expert routing and grouping.
//
// Routing: for each token the topk largest logits (ties to the lowest index),
// weighted by exp(l_j - max) / sum, the sum over the chosen experts
// (renormalised) or over all of them. A logit of -inf or NaN is never chosen:
// a slot left without an expert gets id -1 and weight 0. One warp a token,
// the logits in registers as order-preserving integers; a round of the choice
// is one warp maximum of the keys and one warp minimum of the indices that
// hold it.
//
// Grouping: a stable counting sort of the items (token n, slot j) by id. Each
// block owns a contiguous range of tokens and counts its ids in shared memory
// (integer counts: the order of the atomics does not show). A second kernel
// adds up the counts of the blocks before it and places its items in order,
// 32 at a time, each behind the equal ids on lower lanes. A call of few items
// does all of it in one block of the first kernel.
//
// Bound: a few dependent latencies, not bytes (8191 tokens of 256 bf16
// logits are 4.2 MB, 0.6 us of memory time).
#include <math_constants.h>

#include "moe_internal.cuh"

namespace q6 {
namespace {

constexpr int kRouteThreads = 512;
constexpr int kPlaceThreads = 1024;

// Order-preserving key of a float; 0 (below every key of a number) for -inf
// and NaN. -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (!(x > -CUDART_INF_F)) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// Rows n0..n1-1 of this block.
__device__ __forceinline__ void block_rows(int N, int& n0, int& n1) {
  n0 = (int)((long long)N * blockIdx.x / gridDim.x);
  n1 = (int)((long long)N * (blockIdx.x + 1) / gridDim.x);
}

// The exclusive prefix sum of smem counts cnt[0..G] (G + 1 values) into
// base[0..G], by the whole block; base[G + 1] is the total.
__device__ void block_scan(const int* cnt, int* base, int G) {
  // one warp, 32 counts a step: at most 33 steps
  if (threadIdx.x < 32) {
    int run = 0;
    for (int i0 = 0; i0 <= G; i0 += 32) {
      const int i = i0 + (int)threadIdx.x;
      const int v = i <= G ? cnt[i] : 0;
      int x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if ((int)threadIdx.x >= o) x += y;
      }
      if (i <= G) base[i] = run + x - v;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (threadIdx.x == 0) base[G + 1] = run;
  }
  __syncthreads();
}

// Places the items of rows n0..n1-1 in order: warp 0 takes 32 a step, each
// behind the equal ids on lower lanes; base[g] runs ahead.
__device__ void place_items(const int32_t* ids, int n0, int n1, int per_row, int G, int* base,
                            int32_t* rows, int32_t* pos) {
  if (threadIdx.x >= 32) return;
  const int lane = threadIdx.x;
  const long long i1 = (long long)n1 * per_row;
  for (long long i0 = (long long)n0 * per_row; i0 < i1; i0 += 32) {
    const long long i = i0 + lane;
    int g = -1;
    if (i < i1) {
      g = ids[i];
      if (g < 0 || g >= G) g = G;
    }
    const unsigned same = __match_any_sync(0xffffffffu, g);
    if (g >= 0) {
      const int before = __popc(same & ((1u << lane) - 1u));
      const int at = base[g] + before;
      rows[at] = (int)(i / per_row);
      pos[i] = g < G ? at : -1;
      __syncwarp(same);
      if (before == 0) base[g] += __popc(same);
    }
    __syncwarp();
  }
}

// Ends a counting kernel: a grid of one block scans and places at once, any
// other leaves its counts in hist[block][G + 1].
__device__ void finish_counts(const int32_t* ids, int n0, int n1, int per_row, int G, int* cnt,
                              int* base, int32_t* offsets, int32_t* rows, int32_t* pos,
                              int32_t* hist) {
  if (gridDim.x == 1) {
    block_scan(cnt, base, G);
    for (int g = threadIdx.x; g <= G + 1; g += blockDim.x) offsets[g] = base[g];
    __syncthreads();
    place_items(ids, n0, n1, per_row, G, base, rows, pos);
  } else {
    for (int g = threadIdx.x; g <= G; g += blockDim.x)
      hist[(size_t)blockIdx.x * (G + 1) + g] = cnt[g];
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kRouteThreads)
route_kernel(const T* logits, int N, int E, long long ldl, int topk, int renorm, int32_t* ids,
             float* weights, int32_t* offsets, int32_t* rows, int32_t* pos, int32_t* hist) {
  __shared__ int cnt[kMaxGroups + 1], base[kMaxGroups + 2];
  griddep_wait();
  griddep_launch_dependents();
  for (int g = threadIdx.x; g <= E; g += blockDim.x) cnt[g] = 0;
  __syncthreads();
  int n0, n1;
  block_rows(N, n0, n1);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int n = n0 + warp; n < n1; n += kRouteThreads / 32) {
    const T* row = logits + (size_t)n * ldl;
    uint32_t key[V];
    float x[V];
    bool nan = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * 32 + lane;
      x[v] = e < E ? to_f32(row[e]) : -CUDART_INF_F;
      key[v] = order_key(x[v]);
      nan |= isnan(x[v]);
    }
    float top = 0.0f, sum = 0.0f, mine = 0.0f;
    int my_id = -1;
    for (int j = 0; j < topk; ++j) {
      uint32_t bk = key[0];
      int be = lane;
#pragma unroll
      for (int v = 1; v < V; ++v)
        if (key[v] > bk) {
          bk = key[v];
          be = v * 32 + lane;
        }
      const uint32_t wk = __reduce_max_sync(0xffffffffu, bk);
      if (wk == 0u) break;  // nothing left that can be chosen
      const int we = (int)__reduce_min_sync(0xffffffffu, bk == wk ? (unsigned)be : 0xffffffffu);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v * 32 + lane == we) key[v] = 0u;
      const float l = key_value(wk);
      if (j == 0) top = l;
      const float ex = expf(l - top);
      sum += ex;
      if (lane == j) {
        mine = ex;
        my_id = we;
      }
    }
    if (!renorm) {
      sum = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) sum += expf(x[v] - top);
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (__any_sync(0xffffffffu, nan)) sum = CUDART_NAN_F;  // a NaN logit shows in the weights
    if (lane < topk) {
      const size_t i = (size_t)n * topk + lane;
      ids[i] = my_id;
      weights[i] = my_id < 0 ? 0.0f : mine / sum;
      atomicAdd(&cnt[my_id < 0 ? E : my_id], 1);
    }
  }
  __syncthreads();
  finish_counts(ids, n0, n1, topk, E, cnt, base, offsets, rows, pos, hist);
}

__global__ void __launch_bounds__(kRouteThreads)
count_kernel(const int32_t* ids, int N, int per_row, int G, int32_t* offsets, int32_t* rows,
             int32_t* pos, int32_t* hist) {
  __shared__ int cnt[kMaxGroups + 1], base[kMaxGroups + 2];
  griddep_wait();
  griddep_launch_dependents();
  for (int g = threadIdx.x; g <= G; g += blockDim.x) cnt[g] = 0;
  __syncthreads();
  int n0, n1;
  block_rows(N, n0, n1);
  for (long long i = (long long)n0 * per_row + threadIdx.x; i < (long long)n1 * per_row;
       i += blockDim.x) {
    const int g = ids[i];
    atomicAdd(&cnt[g < 0 || g >= G ? G : g], 1);
  }
  __syncthreads();
  finish_counts(ids, n0, n1, per_row, G, cnt, base, offsets, rows, pos, hist);
}

// The second kernel of a large grouping: this block's first place in every
// group from the counts of all blocks, then its items in order.
__global__ void __launch_bounds__(kPlaceThreads)
place_kernel(const int32_t* ids, int N, int per_row, int G, int32_t* offsets, int32_t* rows,
             int32_t* pos, const int32_t* hist) {
  __shared__ int cnt[kMaxGroups + 1], before[kMaxGroups + 1], base[kMaxGroups + 2];
  for (int g = threadIdx.x; g <= G; g += blockDim.x) cnt[g] = before[g] = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  // several threads a group when there are few groups, each over its share of
  // the blocks
  const int parts = max(1, (int)blockDim.x / (G + 1));
  for (int w = threadIdx.x; w < (G + 1) * parts; w += blockDim.x) {
    const int g = w % (G + 1), p = w / (G + 1);
    const int b1 = (int)((long long)gridDim.x * (p + 1) / parts);
    int all = 0, low = 0;
#pragma unroll 8
    for (int b = (int)((long long)gridDim.x * p / parts); b < b1; ++b) {
      const int c = hist[(size_t)b * (G + 1) + g];
      all += c;
      low += b < (int)blockIdx.x ? c : 0;
    }
    atomicAdd(&cnt[g], all);
    atomicAdd(&before[g], low);
  }
  __syncthreads();
  block_scan(cnt, base, G);
  if (blockIdx.x == 0)
    for (int g = threadIdx.x; g <= G + 1; g += blockDim.x) offsets[g] = base[g];
  __syncthreads();
  for (int g = threadIdx.x; g <= G; g += blockDim.x) base[g] += before[g];
  __syncthreads();
  int n0, n1;
  block_rows(N, n0, n1);
  place_items(ids, n0, n1, per_row, G, base, rows, pos);
}

template <typename T, int V>
cudaError_t route_v(const void* logits, int N, int E, long long ldl, int topk, int renorm,
                    int32_t* ids, float* weights, int32_t* offsets, int32_t* rows, int32_t* pos,
                    int32_t* hist, int blocks, cudaStream_t s) {
  return launch_pdl(route_kernel<T, V>, dim3(blocks), dim3(kRouteThreads), 0, s,
                    static_cast<const T*>(logits), N, E, ldl, topk, renorm, ids, weights, offsets,
                    rows, pos, hist);
}

template <typename T>
cudaError_t route_t(const void* logits, int N, int E, long long ldl, int topk, int renorm,
                    int32_t* ids, float* weights, int32_t* offsets, int32_t* rows, int32_t* pos,
                    int32_t* hist, int blocks, cudaStream_t s) {
#define Q6_ROUTE(V)                                                                             \
  if (E <= 32 * V)                                                                              \
    return route_v<T, V>(logits, N, E, ldl, topk, renorm, ids, weights, offsets, rows, pos,     \
                         hist, blocks, s)
  Q6_ROUTE(1);
  Q6_ROUTE(2);
  Q6_ROUTE(4);
  Q6_ROUTE(8);
  Q6_ROUTE(16);
  Q6_ROUTE(32);
#undef Q6_ROUTE
  return cudaErrorInvalidValue;
}

cudaError_t place(const int32_t* ids, int N, int per_row, int G, int32_t* offsets, int32_t* rows,
                  int32_t* pos, const int32_t* hist, int blocks, cudaStream_t s) {
  return launch_pdl(place_kernel, dim3(blocks), dim3(kPlaceThreads), 0, s, ids, N, per_row, G,
                    offsets, rows, pos, hist);
}

}  // namespace

cudaError_t launch_route(const void* logits, int type, int N, int E, long long ldl, int topk,
                         int renorm, int32_t* ids, float* weights, int32_t* offsets,
                         int32_t* rows, int32_t* pos, int32_t* hist, cudaStream_t s) {
  const int blocks = group_blocks((long long)N * topk, N);
  const cudaError_t e =
      type == Q6_TYPE_F32
          ? route_t<float>(logits, N, E, ldl, topk, renorm, ids, weights, offsets, rows, pos, hist,
                           blocks, s)
      : type == Q6_TYPE_BF16
          ? route_t<__nv_bfloat16>(logits, N, E, ldl, topk, renorm, ids, weights, offsets, rows,
                                   pos, hist, blocks, s)
          : route_t<__half>(logits, N, E, ldl, topk, renorm, ids, weights, offsets, rows, pos,
                            hist, blocks, s);
  if (e != cudaSuccess || blocks == 1) return e;
  return place(ids, N, topk, E, offsets, rows, pos, hist, blocks, s);
}

cudaError_t launch_group(const int32_t* ids, int N, int per_row, int G, int32_t* offsets,
                         int32_t* rows, int32_t* pos, int32_t* hist, cudaStream_t s) {
  const int blocks = group_blocks((long long)N * per_row, N);
  const cudaError_t e = launch_pdl(count_kernel, dim3(blocks), dim3(kRouteThreads), 0, s, ids, N,
                                   per_row, G, offsets, rows, pos, hist);
  if (e != cudaSuccess || blocks == 1) return e;
  return place(ids, N, per_row, G, offsets, rows, pos, hist, blocks, s);
}

}  // namespace q6
