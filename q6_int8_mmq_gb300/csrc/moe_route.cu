// Expert routing and grouping.
//
// Routing: for each token the topk largest logits (ties to the lowest index),
// weighted by exp(l_j - max) / sum, the sum over the chosen experts
// (renormalised) or over all of them. A logit of -inf or NaN is never chosen:
// a slot left without an expert gets id -1 and weight 0. One warp a token,
// the logits in registers as order-preserving integers; a round of the choice
// is one warp maximum of the keys and one warp minimum of the indices that
// hold it. A 16-bit logit and its index make one key, and a round is then one
// add-and-maximum a key and one warp maximum (8191 tokens of 256 logits, topk 8:
// 17.2 us, with two reductions a round 19.1).
//
// Grouping: a stable counting sort of the items (token n, slot j) by id. Each
// block owns a contiguous range of tokens and counts its ids in shared memory
// (integer counts: the order of the atomics does not show). A second kernel
// adds up the counts of the blocks before it and places its items, two threads
// each, behind the equal ids before them in the block (counted one against
// the other in shared memory: 512 items are 32 steps of eight ids). A call of
// few items does all of it in one block of the first kernel.
//
// Bound: integer instructions with many tokens, else a few dependent latencies;
// never bytes (8191 tokens of 256 bf16 logits are 4.2 MB, 0.6 us of memory time,
// and take 16.1 us with topk 8; f32 ones 19.4). One token: 2.9 us out of a graph.
#include <math_constants.h>

#include "moe_internal.cuh"

namespace q6 {
namespace {

constexpr int kPlaceThreads = 1024;
constexpr int kCountThreads = 512;
// Threads of a routing block with V logits a lane (its registers).
template <int V>
constexpr int kRouteThreadsOf = V <= 8 ? 1024 : 512;

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

// The same of a 16-bit logit with its expert below it, so that the largest of a
// warp is one value's maximum (ties: the lowest index); 0 as above.
template <typename T>
__device__ __forceinline__ uint32_t packed_key(T v, int e) {
  if (!(to_f32(v) > -CUDART_INF_F)) return 0u;
  uint32_t u = *reinterpret_cast<const uint16_t*>(&v);
  if (u == 0x8000u) u = 0u;
  return (u ^ (u >> 15 ? 0xFFFFu : 0x8000u)) << 16 | (0xFFFFu - (uint32_t)e);
}
__device__ __forceinline__ int packed_expert(uint32_t k) { return (int)(0xFFFFu - (k & 0xFFFFu)); }
template <typename T>
__device__ __forceinline__ float packed_value(uint32_t k) {
  const uint16_t u = (uint16_t)((k >> 16) ^ (k >> 31 ? 0x8000u : 0xFFFFu));
  return to_f32(*reinterpret_cast<const T*>(&u));
}

// Rows n0..n1-1 of this block.
__device__ __forceinline__ void block_rows(int N, int& n0, int& n1) {
  n0 = (int)((long long)N * blockIdx.x / gridDim.x);
  n1 = (int)((long long)N * (blockIdx.x + 1) / gridDim.x);
}

// The exclusive prefix sum of smem counts cnt[0..G] (G + 1 values) into
// base[0..G], by the whole block; base[G + 1] is the total.
__device__ void block_scan(const int* cnt, int* base, int G) {
  __shared__ int warps[32];
  const int per = (G + (int)blockDim.x) / (int)blockDim.x;  // consecutive values a thread
  const int i0 = (int)threadIdx.x * per, i1 = min(i0 + per, G + 1);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int mine = 0;
  for (int i = i0; i < i1; ++i) mine += cnt[i];
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  int before = x - mine;
  for (int w = 0; w < warp; ++w) before += warps[w];
  for (int i = i0; i < i1; ++i) {
    base[i] = before;
    before += cnt[i];
  }
  if (threadIdx.x == blockDim.x - 1) base[G + 1] = before;
  __syncthreads();
}

// Places the items of rows n0..n1-1 in order, blockDim.x / 2 at a time, two
// threads an item; base[g] runs ahead. ids_s holds that many ids.
__device__ void place_items(const int32_t* ids, int n0, int n1, int per_row, int G, int* base,
                            int* ids_s, int32_t* rows, int32_t* pos) {
  const int me = threadIdx.x / 2, half = threadIdx.x % 2, chunk = (int)blockDim.x / 2;
  const long long end = (long long)n1 * per_row;
  for (long long i0 = (long long)n0 * per_row; i0 < end; i0 += chunk) {
    const long long i = i0 + me;
    int g = -1;
    if (i < end) {
      g = ids[i];
      if (g < 0 || g >= G) g = G;
    }
    if (half == 0) ids_s[me] = g;
    __syncthreads();
    // equal ids before mine: whole groups of eight, every other one by each of
    // the two threads, then what is left
    int before = 0;
    if (g >= 0) {
      const int4* v = reinterpret_cast<const int4*>(ids_s);
      for (int k = half; k < me / 8; k += 2) {
        const int4 a = v[2 * k], b = v[2 * k + 1];
        before += (a.x == g) + (a.y == g) + (a.z == g) + (a.w == g) + (b.x == g) + (b.y == g) +
                  (b.z == g) + (b.w == g);
      }
      for (int k = me / 8 * 8 + half; k < me; k += 2) before += ids_s[k] == g;
    }
    before += __shfl_xor_sync(0xffffffffu, before, 1);
    int at = 0;
    if (g >= 0) at = base[g] + before;
    __syncthreads();
    if (g >= 0 && half == 0) {
      rows[at] = (int)(i / per_row);
      pos[i] = g < G ? at : -1;
      if (i0 + chunk < end) atomicAdd(&base[g], 1);
    }
    if (i0 + chunk < end) __syncthreads();
  }
}

// Ends a counting kernel: a grid of one block scans and places at once, any
// other leaves its counts in hist[block][G + 1].
__device__ void finish_counts(const int32_t* ids, int n0, int n1, int per_row, int G, int* cnt,
                              int* base, int* ids_s, int32_t* offsets, int32_t* rows,
                              int32_t* pos, int32_t* hist) {
  if (gridDim.x == 1) {
    block_scan(cnt, base, G);
    for (int g = threadIdx.x; g <= G + 1; g += blockDim.x) offsets[g] = base[g];
    __syncthreads();
    place_items(ids, n0, n1, per_row, G, base, ids_s, rows, pos);
  } else {
    const int ld = group_hist_ld(G);  // past G: zeros
    for (int g = threadIdx.x; g < ld; g += blockDim.x)
      hist[(size_t)blockIdx.x * ld + g] = g <= G ? cnt[g] : 0;
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kRouteThreadsOf<V>)
route_kernel(const T* logits, int N, int E, long long ldl, int topk, int renorm, int32_t* ids,
             float* weights, int32_t* offsets, int32_t* rows, int32_t* pos, int32_t* hist) {
  __shared__ int cnt[kMaxGroups + 1], base[kMaxGroups + 2];
  __shared__ __align__(16) int ids_s[512];
  griddep_wait();
  griddep_launch_dependents();
  for (int g = threadIdx.x; g <= E; g += blockDim.x) cnt[g] = 0;
  __syncthreads();
  int n0, n1;
  block_rows(N, n0, n1);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int n = n0 + warp; n < n1; n += (int)blockDim.x / 32) {
    const T* row = logits + (size_t)n * ldl;
    constexpr bool kPacked = sizeof(T) == 2;
    uint32_t key[V];
    bool nan = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * 32 + lane;
      const T x = e < E ? row[e] : from_f32<T>(-CUDART_INF_F);
      if constexpr (kPacked) {
        key[v] = packed_key(x, e);
      } else {
        key[v] = order_key(x);
      }
      nan |= isnan(to_f32(x));
    }
    float top = 0.0f, mine = 0.0f;
    int my_id = -1;
    uint32_t last = 0u;  // packed: what was chosen last
    for (int j = 0; j < topk; ++j) {
      int we;
      float l;
      if constexpr (kPacked) {
        // the largest key below the last one: key - last modulo 2^32 is larger
        // for keys below it than for all others (and for last = 0 the key itself)
        uint32_t most = 0u;
#pragma unroll
        for (int v = 0; v < V; ++v) most = __viaddmax_u32(key[v], 0u - last, most);
        const uint32_t wk = __reduce_max_sync(0xffffffffu, most) + last;
        if (wk == 0u || (last != 0u && wk >= last)) break;  // nothing left that can be chosen
        last = wk;
        we = packed_expert(wk);
        l = packed_value<T>(wk);
      } else {
        uint32_t bk = key[0];
        int be = lane;
#pragma unroll
        for (int v = 1; v < V; ++v)
          if (key[v] > bk) {
            bk = key[v];
            be = v * 32 + lane;
          }
        const uint32_t wk = __reduce_max_sync(0xffffffffu, bk);
        if (wk == 0u) break;
        we = (int)__reduce_min_sync(0xffffffffu, bk == wk ? (unsigned)be : 0xffffffffu);
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (v * 32 + lane == we) key[v] = 0u;
        l = key_value(wk);
      }
      if (j == 0) top = l;
      if (lane == j) {
        mine = l;
        my_id = we;
      }
    }
    mine = my_id < 0 ? 0.0f : expf(mine - top);  // this lane's slot
    float sum = mine;
    if (!renorm) {
      sum = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = v * 32 + lane;
        sum += expf((e < E ? to_f32(row[e]) : -CUDART_INF_F) - top);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (__any_sync(0xffffffffu, nan)) sum = CUDART_NAN_F;  // a NaN logit shows in the weights
    if (lane < topk) {
      const size_t i = (size_t)n * topk + lane;
      ids[i] = my_id;
      weights[i] = my_id < 0 ? 0.0f : mine / sum;
      atomicAdd(&cnt[my_id < 0 ? E : my_id], 1);
    }
  }
  __syncthreads();
  finish_counts(ids, n0, n1, topk, E, cnt, base, ids_s, offsets, rows, pos, hist);
}

__global__ void __launch_bounds__(kCountThreads)
count_kernel(const int32_t* ids, int N, int per_row, int G, int32_t* offsets, int32_t* rows,
             int32_t* pos, int32_t* hist) {
  __shared__ int cnt[kMaxGroups + 1], base[kMaxGroups + 2];
  __shared__ __align__(16) int ids_s[512];
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
  finish_counts(ids, n0, n1, per_row, G, cnt, base, ids_s, offsets, rows, pos, hist);
}

// The second kernel of a large grouping: this block's first place in every
// group from the counts of all blocks, then its items in order.
__global__ void __launch_bounds__(kPlaceThreads)
place_kernel(const int32_t* ids, int N, int per_row, int G, int32_t* offsets, int32_t* rows,
             int32_t* pos, const int32_t* hist) {
  __shared__ int cnt[kMaxGroups + 4], before[kMaxGroups + 4], base[kMaxGroups + 2];
  __shared__ __align__(16) int ids_s[kPlaceThreads / 2];
  const int ld = group_hist_ld(G);
  for (int g = threadIdx.x; g < ld; g += blockDim.x) cnt[g] = before[g] = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  // four groups a thread, several threads for the same four, each over its
  // share of the blocks
  const int quads = ld / 4, parts = max(1, (int)blockDim.x / quads);
  for (int w = threadIdx.x; w < quads * parts; w += blockDim.x) {
    const int q = w % quads, p = w / quads;
    const int b1 = (int)gridDim.x * (p + 1) / parts;
    int all[4] = {}, low[4] = {};
#pragma unroll 8
    for (int b = (int)gridDim.x * p / parts; b < b1; ++b) {
      const int4 c = *reinterpret_cast<const int4*>(hist + (size_t)b * ld + 4 * q);
      const int m = b < (int)blockIdx.x ? -1 : 0;
      all[0] += c.x, all[1] += c.y, all[2] += c.z, all[3] += c.w;
      low[0] += c.x & m, low[1] += c.y & m, low[2] += c.z & m, low[3] += c.w & m;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (all[k]) atomicAdd(&cnt[4 * q + k], all[k]);
      if (low[k]) atomicAdd(&before[4 * q + k], low[k]);
    }
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
  place_items(ids, n0, n1, per_row, G, base, ids_s, rows, pos);
}

template <typename T, int V>
cudaError_t route_v(const void* logits, int N, int E, long long ldl, int topk, int renorm,
                    int32_t* ids, float* weights, int32_t* offsets, int32_t* rows, int32_t* pos,
                    int32_t* hist, int blocks, cudaStream_t s) {
  // a warp a token where one block has few
  const int threads = blocks == 1 && N < kRouteThreadsOf<V> / 32 ? (N < 4 ? 128 : 32 * N)
                                                                 : kRouteThreadsOf<V>;
  return launch_pdl(route_kernel<T, V>, dim3(blocks), dim3(threads), 0, s,
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
  const cudaError_t e = launch_pdl(count_kernel, dim3(blocks), dim3(kCountThreads), 0, s, ids, N,
                                   per_row, G, offsets, rows, pos, hist);
  if (e != cudaSuccess || blocks == 1) return e;
  return place(ids, N, per_row, G, offsets, rows, pos, hist, blocks, s);
}

}  // namespace q6
