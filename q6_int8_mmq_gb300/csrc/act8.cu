// Activations quantised by the step that makes them: the root-mean-square norm
// with the residual's addition, silu(gate) * up, or (e4m3 alone; the int8 codes of f32
// rows are quantize.cu's) nothing but the reading.
//
//   norm   h = x + residual,  t = h * weight,  r = 1 / sqrt(mean(h^2) + eps)
//   silu   t = gate / (1 + exp(-gate)) * up,   r = 1
//   rows   t = x,                              r = 1
//   int8   per 32:  d = max|t| / 127, code = round(t / d), halves away from 0;
//                   scale r * d
//   e4m3   per 128: d = max|t| / 448, code = e4m3(t * (448 / max|t|)); scale r * d
//
// Bound: memory. (us and share of what a plain copy reaches: the norm of 8192 x 4096
// bf16 with a bf16 residual 39.9, 87 %; of 3314 x 4096 f32 to int8 36.0, 84 %; silu(gate)
// * up of 3314 x 11008 f32 to int8 58.9, 92 %; a weight of 11008 x 4096 bf16 23.4, 85 %.)
//
// The norm's 1 / rms is one factor for a whole row, so it goes into the row's
// scales and the codes do not wait for it: the row is read once, its codes are
// written as it is read, and what is kept until the sum of squares is there is
// one number a block.
//
// A block that holds an infinity or a NaN gets codes 0 and a NaN scale; an e4m3
// block whose largest value is below 2^-100 codes and scale 0.
#include "f8_internal.cuh"
#include "q6_quant.cuh"

namespace q6 {
namespace {

constexpr float kF8Max = 448.0f, kF8Tiny = 0x1p-100f;

// A thread's kPer (8 or 16) consecutive values as they lie in memory (16-byte
// aligned), and as f32. A block's scale costs two divisions or a division and a
// reciprocal, about 40 instructions, so it is worth 16 values a thread (with 8, e4m3
// codes of 3325 x 3584 binary16 values take 10.3 instead of 8.5 us); but not for
// int8 codes of f32 rows, where a thread's loads would lie 64 bytes apart (the norm
// of 3314 x 4096: 42.9 instead of 34.6 us). e4m3 codes of f32 rows take 16 all the same;
// 8 have not been measured there. (3314 x 4096, us and share of a copy's rate: the norm
// of f32 with an f32 residual 37.0, 70 %, bf16 with f32 31.9, 69 %, f32 with bf16 25.2, 71 %;
// silu(gate) * up of 3314 x 11008 49.5, 98 %; the quantiser of 3325 x 3584 10.8, 82 %.)
template <typename T, int kPer>
struct Raw {
  static constexpr int kLoads = kPer * (int)sizeof(T) / 16;
  uint4 u[kLoads];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void get(float (&v)[kPer]) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          v[4 * i + j] = __uint_as_float(w[j]);
        } else {
          const float2 f = unpack2<T>(w[j]);
          v[8 * i + 2 * j] = f.x, v[8 * i + 2 * j + 1] = f.y;
        }
      }
    }
  }
  static __device__ __forceinline__ void store(T* p, const float (&v)[kPer]) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(v[4 * i + j]);
        else w[j] = pack2<T>(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
      }
      reinterpret_cast<uint4*>(p)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};
// The same of a type known at run time (the norm's weight).
template <typename T, int kPer>
__device__ __forceinline__ void load_as(const void* p, size_t at, float (&v)[kPer]) {
  Raw<T, kPer> r;
  r.load(static_cast<const T*>(p) + at);
  r.get(v);
}
template <int kPer>
__device__ __forceinline__ void load_of(const void* p, int type, size_t at, float (&v)[kPer]) {
  if (type == Q6_TYPE_F32) load_as<float>(p, at, v);
  else if (type == Q6_TYPE_BF16) load_as<__nv_bfloat16>(p, at, v);
  else load_as<__half>(p, at, v);
}

// The larger one; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
template <int kPer>
__device__ __forceinline__ float largest(const float (&v)[kPer]) {
  float a = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < kPer; ++i) a = max_nan(a, fabsf(v[i]));
  return a;
}
template <int kLanes>
__device__ __forceinline__ float group_max(float a) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}
// Two values -> their e4m3 codes, a in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float nan_f32() { return __uint_as_float(0x7FC00000u); }

// A block's scale without the row's factor, and what its values are multiplied with
// (e4m3: 448 / largest; int8: the reciprocal of the scale, which comes with it).
// Called by whole warps whose neighbouring lanes have the same block.
struct Scale {
  float d, by;
  bool fine;  // no infinity, no NaN
};
template <bool kF8>
__device__ __forceinline__ Scale scale_of(float top) {
  Scale s;
  s.fine = top < __uint_as_float(0x7F800000u);
  if constexpr (kF8) {
    // both quotients by one division: 448 / top in even lanes, top / 448 in odd ones
    const bool odd = threadIdx.x & 1;
    const float q = __fdiv_rn(odd ? top : kF8Max, odd ? kF8Max : top);
    const float p = __shfl_xor_sync(0xffffffffu, q, 1);
    const bool live = s.fine && top >= kF8Tiny;
    s.d = !s.fine ? nan_f32() : live ? (odd ? q : p) : 0.0f;
    s.by = live ? (odd ? p : q) : 0.0f;
  } else {
    s.d = s.fine ? __fdiv_rn(top, 127.0f) : nan_f32();
    s.by = recip_or_zero(s.d);  // 0 for NaN
  }
  return s;
}
// kPer values of a block -> their codes at element `at` of the output rows.
// Returns the sum of int8 codes.
template <bool kF8, int kPer>
__device__ __forceinline__ float store_codes(const RowSink& o, size_t at, float (&v)[kPer],
                                             const Scale& s) {
  if (!s.fine) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = 0.0f;
  }
  if constexpr (kF8) {
    uint32_t c[kPer / 4];
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i)
      c[i] = e4m3x2(v[4 * i] * s.by, v[4 * i + 1] * s.by) |
             e4m3x2(v[4 * i + 2] * s.by, v[4 * i + 3] * s.by) << 16;
    if constexpr (kPer == 16) *reinterpret_cast<uint4*>(o.q + at) = make_uint4(c[0], c[1], c[2], c[3]);
    else *reinterpret_cast<uint2*>(o.q + at) = make_uint2(c[0], c[1]);
    return 0.0f;
  } else {
    const float d = s.fine ? s.d : 0.0f;
    uint2 q[kPer / 8];
    uint4 h[kPer / 8];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kPer / 8; ++j) {
      const float* t = v + 8 * j;
      float part;
      quant8_sum(make_float4(t[0], t[1], t[2], t[3]), make_float4(t[4], t[5], t[6], t[7]), d, s.by,
                 q[j], h[j], part);
      sum += part;
    }
    if (o.q) {
      if constexpr (kPer == 16)
        *reinterpret_cast<uint4*>(o.q + at) = make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
      else
        *reinterpret_cast<uint2*>(o.q + at) = q[0];
    }
    if (o.xh) {
#pragma unroll
      for (int j = 0; j < kPer / 8; ++j) reinterpret_cast<uint4*>(o.xh + at)[j] = h[j];
    }
    return sum;
  }
}

template <bool kF8>
constexpr int kBlock = kF8 ? kF8Block : kQ8Block;
// Of a kernel: a thread's values, the threads of a block, a warp's part of a row.
template <bool kF8, int kBytes>
struct Shape {
  static constexpr int kPer = kF8 || kBytes == 2 ? 16 : 8;
  static constexpr int kLanes = kBlock<kF8> / kPer, kPart = 32 * kPer;
  // the sum of a block's lanes
  static __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
};

// x / (1 + exp(-x)): the exponential's 2 + 1.2 |x| and the division's 2 units of 2^-23.
__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.0f + __expf(-x)); }

// CTAs an SM: what is in flight is bytes a thread times threads, so registers are
// held to 48 for up to 64 bytes, to 64 for more (silu(gate) * up of 3314 x 11008, us:
// bf16 to int8 51.5 with 66 registers, 44.5; to e4m3 34.0, 33.0; f32 to int8 62.7,
// 58.9. With 40 registers 57.6 for the first). 12 of the 17 forms spill 16 to 108 bytes at
// these limits, those three 56, 16 and 36, and are the faster for it.
template <typename T, bool kF8, bool kGlu, int kU>
constexpr int kRowCtas =
    Shape<kF8, (int)sizeof(T)>::kPer * (int)sizeof(T) * (kGlu ? 2 : 1) * kU <= 64 ? 5 : 4;

// Rows without a factor: a warp takes kU parts of a row at a time,
// their loads in flight together.
template <typename T, bool kF8, bool kGlu, int kU>
__global__ void __launch_bounds__(256, kRowCtas<T, kF8, kGlu, kU>) rows_kernel(const T* X, int N, int K, long long ldx,
                                                   const RowSink o) {
  using S = Shape<kF8, (int)sizeof(T)>;
  constexpr int kPer = S::kPer, kLanes = S::kLanes, kPartK = S::kPart;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, tasks = (K + kPartK * kU - 1) / (kPartK * kU);  // of a row
  const long long total = (long long)N * tasks;
  const long long step = (long long)gridDim.x * 8;
  for (long long g = (long long)blockIdx.x * 8 + threadIdx.x / 32; g < total; g += step) {
    const int n = total < 1ll << 31 ? (int)g / tasks : (int)(g / tasks);
    const int first = (int)(g - (long long)n * tasks) * (kPartK * kU), k0 = first + kPer * lane;
    const T* x = X + n * ldx + k0;
    Raw<T, kPer> raw[kU], up[kGlu ? kU : 1];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (k0 + kPartK * u < K) {
        raw[u].load(x + kPartK * u);
        if constexpr (kGlu) up[u].load(x + K + kPartK * u);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int k = k0 + kPartK * u;
      if (kU > 1 && first + kPartK * u >= K) break;
      float v[kPer] = {};
      if (k < K) {
        raw[u].get(v);
        if constexpr (kGlu) {
          float w[kPer];
          up[u].get(w);
#pragma unroll
          for (int i = 0; i < kPer; ++i) v[i] = silu(v[i]) * w[i];
        }
      }
      const Scale s = scale_of<kF8>(group_max<kLanes>(largest(v)));
      float sum = 0.0f;
      if (k < K) sum = store_codes<kF8>(o, (size_t)n * K + k, v, s);
      if (!kF8 && o.us) sum = S::sum(sum);
      if (k < K && lane % kLanes == 0) {
        const int b = k / kBlock<kF8>;
        o.scale[(size_t)b * o.lds + n] = s.d;
        if (!kF8 && o.us) store_us(o.us, n, K, b, s.d * sum);
      }
    }
  }
}

// One row a CTA, kU parts a warp in flight together. The scales (and for us the sums)
// of its blocks wait in shared memory for the row's factor. (At most 85 registers: with
// 64 the norm of 8192 x 4096 bf16 takes 48.4 instead of 39.7 us, unbound 42.2. e4m3 codes
// with an f32 X or residual spill at that limit, 112 bytes where both are, else 32 or 48;
// with a part a warp 16 to 32.)
template <typename T, typename R, bool kF8, bool kAdd, int kU>
__global__ void __launch_bounds__(kU > 1 ? 256 : 1024, kU > 1 ? 3 : 1) norm_kernel(const NormCall c, const RowSink o) {
  using S = Shape<kF8, (int)(sizeof(T) > sizeof(R) ? sizeof(T) : sizeof(R))>;
  constexpr int kPer = S::kPer, kLanes = S::kLanes, kPartK = S::kPart;
  extern __shared__ float kept[];
  __shared__ float parts[32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, K = c.K;
  const int blocks = (K + kBlock<kF8> - 1) / kBlock<kF8>;
  const size_t n = blockIdx.x;
  const T* x = static_cast<const T*>(c.X) + n * c.ldx;
  const R* res = static_cast<const R*>(c.residual) + n * c.ldr;
  R* hout = static_cast<R*>(c.h) + n * c.ldh;
  float squares = 0.0f;
  for (int k0 = warp * kPartK * kU; k0 < K; k0 += (blockDim.x >> 5) * kPartK * kU) {
    Raw<T, kPer> raw[kU];
    Raw<R, kPer> rest[kAdd ? kU : 1];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int k = k0 + kPartK * u + kPer * lane;
      if (k < K) {
        raw[u].load(x + k);
        if constexpr (kAdd) rest[u].load(res + k);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (kU > 1 && k0 + kPartK * u >= K) break;
      const int k = k0 + kPartK * u + kPer * lane;
      float v[kPer] = {};
      if (k < K) {
        raw[u].get(v);
        if constexpr (kAdd) {
          float r[kPer];
          rest[u].get(r);
#pragma unroll
          for (int i = 0; i < kPer; ++i) v[i] += r[i];
          Raw<R, kPer>::store(hout + k, v);
        }
        float w[kPer];
        load_of(c.weight, c.wtype, k, w);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          squares = fmaf(v[i], v[i], squares);
          v[i] *= w[i];
        }
      }
      const Scale s = scale_of<kF8>(group_max<kLanes>(largest(v)));
      float sum = 0.0f;
      if (k < K) sum = store_codes<kF8>(o, n * K + k, v, s);
      if (!kF8 && o.us) sum = S::sum(sum);
      if (k < K && lane % kLanes == 0) {
        const int b = k / kBlock<kF8>;
        kept[b] = s.d;
        if (!kF8 && o.us) kept[blocks + b] = sum;
      }
    }
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) squares += __shfl_xor_sync(0xffffffffu, squares, s);
  if (lane == 0) parts[warp] = squares;
  __syncthreads();
  float total = 0.0f;
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) total += parts[i];
  const float root = __frsqrt_rn(total / (float)K + c.eps);
  for (int b = threadIdx.x; b < blocks; b += blockDim.x) {
    const float d = root * kept[b];
    o.scale[(size_t)b * o.lds + n] = d;
    if (!kF8 && o.us) store_us(o.us, (int)n, K, b, d * kept[blocks + b]);
  }
}

// One block of 128 x 128 a CTA: a warp takes four rows at a time, and keeps them as
// they came until the block's largest value is known. (16-bit weights spill 104 bytes at
// the 64 registers of four CTAs an SM.)
template <typename T>
__global__ void __launch_bounds__(256, sizeof(T) == 4 ? 2 : 4) weights_kernel(const T* W, int M, int K, long long ldw,
                                                      uint8_t* wq, float* sw) {
  __shared__ float tops[8];
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kPer = 16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int across = (K + kF8Block - 1) / kF8Block;
  const int mb = blockIdx.x / across, kb = blockIdx.x - mb * across;
  const int k = kb * kF8Block + kPer * (lane & 7);
  const long long m0 = (long long)mb * kF8Block + 4 * warp + (lane >> 3);
  Raw<T, kPer> raw[4] = {};
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long m = m0 + 32 * i;
    if (m < M && k < K) raw[i].load(W + m * ldw + k);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[kPer];
    raw[i].get(v);
    top = max_nan(top, largest(v));
  }
  top = group_max<32>(top);
  if (lane == 0) tops[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_nan(top, tops[i]);
  const Scale s = scale_of<true>(top);
  RowSink o = {};
  o.q = wq;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long m = m0 + 32 * i;
    float v[kPer];
    raw[i].get(v);
    if (m < M && k < K) store_codes<true>(o, (size_t)m * K + k, v, s);
  }
  if (threadIdx.x == 0) sw[blockIdx.x] = s.d;
}

template <typename T, bool kF8, bool kGlu, int kU>
cudaError_t rows_u(const void* X, int N, int K, long long ldx, const RowSink& out, cudaStream_t s) {
  constexpr int kTask = Shape<kF8, (int)sizeof(T)>::kPart * kU;
  const long long tasks = (long long)N * (((long long)K + kTask - 1) / kTask);
  const long long blocks = (tasks + 7) / 8;
  const unsigned grid = (unsigned)(blocks < 152 * 32 ? blocks : 152 * 32);
  return launch_pdl(rows_kernel<T, kF8, kGlu, kU>, dim3(grid), dim3(256), 0, s,
                    static_cast<const T*>(X), N, K, ldx, out);
}
// Up to 128 bytes of a thread in flight where there are parts enough for all SMs.
template <typename T, bool kF8, bool kGlu>
cudaError_t rows_t(const void* X, int N, int K, long long ldx, const RowSink& out, cudaStream_t s) {
  using S = Shape<kF8, (int)sizeof(T)>;
  constexpr int kBytes = S::kPer * (int)sizeof(T) * (kGlu ? 2 : 1), kU = kBytes < 128 ? 128 / kBytes : 1;
  if (kU > 1 && (long long)N * K >= 152ll * 8 * S::kPart * kU)
    return rows_u<T, kF8, kGlu, kU>(X, N, K, ldx, out, s);
  return rows_u<T, kF8, kGlu, 1>(X, N, K, ldx, out, s);
}
template <bool kF8, bool kGlu>
cudaError_t rows_as(const void* X, int type, int N, int K, long long ldx, const RowSink& out,
                    cudaStream_t s) {
  return type == Q6_TYPE_F32    ? rows_t<float, kF8, kGlu>(X, N, K, ldx, out, s)
         : type == Q6_TYPE_BF16 ? rows_t<__nv_bfloat16, kF8, kGlu>(X, N, K, ldx, out, s)
                                : rows_t<__half, kF8, kGlu>(X, N, K, ldx, out, s);
}

template <typename T, typename R, bool kF8, bool kAdd, int kU>
cudaError_t norm_u(const NormCall& c, const RowSink& out, int most, cudaStream_t s) {
  constexpr int kTask = Shape<kF8, (int)(sizeof(T) > sizeof(R) ? sizeof(T) : sizeof(R))>::kPart * kU;
  int threads = (c.K + kTask - 1) / kTask * 32;
  if (threads > most) threads = most;
  const int blocks = (c.K + kBlock<kF8> - 1) / kBlock<kF8>;
  const size_t smem = (size_t)blocks * (out.us ? 8 : 4);
  return launch_pdl(norm_kernel<T, R, kF8, kAdd, kU>, dim3((unsigned)c.N), dim3((unsigned)threads),
                    smem, s, c, out);
}
// Few rows: a part a warp, all of a row's loads at once. Many: two parts a warp and 256
// threads a row, so that more rows share an SM (8192 x 4096 bf16 39.9 us, with one part
// 43.3; but 512 x 4096 5.5, with one 4.8).
template <typename T, typename R, bool kF8, bool kAdd>
cudaError_t norm_t(const NormCall& c, const RowSink& out, cudaStream_t s) {
  if (c.N <= 152) return norm_u<T, R, kF8, kAdd, 1>(c, out, 1024, s);
  if ((long long)c.N * c.K < 1ll << 23) return norm_u<T, R, kF8, kAdd, 1>(c, out, 256, s);
  return norm_u<T, R, kF8, kAdd, 2>(c, out, 256, s);
}
template <typename T, typename R, bool kAdd>
cudaError_t norm_as(const NormCall& c, const RowSink& out, cudaStream_t s) {
  return out.f8 ? norm_t<T, R, true, kAdd>(c, out, s) : norm_t<T, R, false, kAdd>(c, out, s);
}
template <typename T>
cudaError_t norm_of(const NormCall& c, const RowSink& out, cudaStream_t s) {
  if (!c.residual) return norm_as<T, T, false>(c, out, s);
  return c.rtype == Q6_TYPE_F32    ? norm_as<T, float, true>(c, out, s)
         : c.rtype == Q6_TYPE_BF16 ? norm_as<T, __nv_bfloat16, true>(c, out, s)
                                   : norm_as<T, __half, true>(c, out, s);
}
template <typename T>
cudaError_t weights_t(const void* W, int M, int K, long long ldw, uint8_t* wq, float* sw,
                      cudaStream_t s) {
  return launch_pdl(weights_kernel<T>, dim3((unsigned)f8_blocks(M) * (unsigned)f8_blocks(K)),
                    dim3(256), 0, s, static_cast<const T*>(W), M, K, ldw, wq, sw);
}

}  // namespace

cudaError_t launch_f8_quantize_rows(const void* X, int type, int N, int K, long long ldx,
                                    const RowSink& out, cudaStream_t s) {
  return rows_as<true, false>(X, type, N, K, ldx, out, s);
}
cudaError_t launch_silu_mul(const void* X, int type, int N, int K, long long ldx,
                            const RowSink& out, cudaStream_t s) {
  return out.f8 ? rows_as<true, true>(X, type, N, K, ldx, out, s)
                : rows_as<false, true>(X, type, N, K, ldx, out, s);
}
cudaError_t launch_rms_norm(const NormCall& c, const RowSink& out, cudaStream_t s) {
  return c.type == Q6_TYPE_F32    ? norm_of<float>(c, out, s)
         : c.type == Q6_TYPE_BF16 ? norm_of<__nv_bfloat16>(c, out, s)
                                  : norm_of<__half>(c, out, s);
}
cudaError_t launch_f8_quantize_weights(const void* W, int type, int M, int K, long long ldw,
                                       uint8_t* wq, float* sw, cudaStream_t s) {
  return type == Q6_TYPE_F32    ? weights_t<float>(W, M, K, ldw, wq, sw, s)
         : type == Q6_TYPE_BF16 ? weights_t<__nv_bfloat16>(W, M, K, ldw, wq, sw, s)
                                : weights_t<__half>(W, M, K, ldw, wq, sw, s);
}

}  // namespace q6
