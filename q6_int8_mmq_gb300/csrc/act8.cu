// Activations quantised by the step that makes them: the root-mean-square norm
// with the residual's addition, silu(gate) * up, or nothing but the reading.
//
//   norm   h = x + residual,  t = h * weight,  r = 1 / sqrt(mean(h^2) + eps)
//   silu   t = gate / (1 + exp(-gate)) * up,   r = 1
//   rows   t = x,                              r = 1
//   int8   per 32:  d = max|t| / 127, code = round(t / d), halves away from 0;
//                   scale r * d
//   e4m3   per 128: d = max|t| / 448, code = e4m3(t * (448 / max|t|)); scale r * d
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

// Eight consecutive values as f32 (16-byte aligned).
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<T>(w[i]);
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]),
                                            pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
// Eight values of a type known at run time (the norm's weight).
__device__ __forceinline__ void load8_of(const void* p, int type, size_t at, float (&v)[8]) {
  if (type == Q6_TYPE_F32) load8(static_cast<const float*>(p) + at, v);
  else if (type == Q6_TYPE_BF16) load8(static_cast<const __nv_bfloat16*>(p) + at, v);
  else load8(static_cast<const __half*>(p) + at, v);
}

// The larger one; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float largest8(const float (&v)[8]) {
  float a = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) a = max_nan(a, fabsf(v[i]));
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

// Eight values of a block whose largest is `top` -> their codes at element `at`
// of the output rows.
template <bool kF8>
__device__ __forceinline__ float store_codes(const RowSink& o, size_t at, float (&v)[8], float top) {
  float sum = 0.0f;
  const bool fine = top < __uint_as_float(0x7F800000u);
  if constexpr (kF8) {
    const float up = fine && top >= kF8Tiny ? __fdiv_rn(kF8Max, top) : 0.0f;
    if (!fine) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    }
    uint2 c;
    c.x = e4m3x2(v[0] * up, v[1] * up) | e4m3x2(v[2] * up, v[3] * up) << 16;
    c.y = e4m3x2(v[4] * up, v[5] * up) | e4m3x2(v[6] * up, v[7] * up) << 16;
    *reinterpret_cast<uint2*>(o.q + at) = c;
  } else {
    float d = __fdiv_rn(top, 127.0f);
    if (!fine) {
      d = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    }
    uint2 q8;
    uint4 h8;
    quant8_sum(make_float4(v[0], v[1], v[2], v[3]), make_float4(v[4], v[5], v[6], v[7]), d,
               recip_or_zero(d), q8, h8, sum);
    if (o.q) *reinterpret_cast<uint2*>(o.q + at) = q8;
    if (o.xh) *reinterpret_cast<uint4*>(o.xh + at) = h8;
  }
  return sum;
}
// A block's scale from its largest value, without the row's factor.
template <bool kF8>
__device__ __forceinline__ float block_scale(float top) {
  if (!(top < __uint_as_float(0x7F800000u))) return nan_f32();
  if constexpr (kF8) return top >= kF8Tiny ? __fdiv_rn(top, kF8Max) : 0.0f;
  return __fdiv_rn(top, 127.0f);
}

template <bool kF8>
constexpr int kLanes = (kF8 ? kF8Block : kQ8Block) / 8;  // threads of a block

// x / (1 + exp(-x)): the exponential's 2 + 1.2 |x| and the division's 2 units of 2^-23.
__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.0f + __expf(-x)); }

// Rows without a factor: a warp takes 256 elements of a row at a time.
template <typename T, bool kF8, bool kGlu>
__global__ void __launch_bounds__(256) rows_kernel(const T* X, int N, int K, long long ldx,
                                                   const RowSink o) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, parts = (K + 255) / 256;
  const long long total = (long long)N * parts;
  const long long step = (long long)gridDim.x * 8;
  for (long long g = (long long)blockIdx.x * 8 + threadIdx.x / 32; g < total; g += step) {
    const int n = (int)(g / parts), k = (int)(g - (long long)n * parts) * 256 + 8 * lane;
    float v[8] = {};
    if (k < K) {
      load8(X + n * ldx + k, v);
      if constexpr (kGlu) {
        float u[8];
        load8(X + n * ldx + K + k, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = silu(v[i]) * u[i];
      }
    }
    const float top = group_max<kLanes<kF8>>(largest8(v));
    float sum = 0.0f;
    if (k < K) sum = store_codes<kF8>(o, (size_t)n * K + k, v, top);
    if (!kF8 && o.us) {
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    }
    if (k < K && lane % kLanes<kF8> == 0) {
      const int b = k / (8 * kLanes<kF8>);
      const float d = block_scale<kF8>(top);
      o.scale[(size_t)b * o.lds + n] = d;
      if (!kF8 && o.us) store_us(o.us, n, K, b, d * sum);
    }
  }
}

// One row a CTA. tops (and for us sums) of its blocks wait in shared memory.
template <typename T, typename R, bool kF8, bool kAdd>
__global__ void __launch_bounds__(1024) norm_kernel(const NormCall c, const RowSink o) {
  extern __shared__ float kept[];
  __shared__ float parts[32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, K = c.K;
  const int blocks = (K + 8 * kLanes<kF8> - 1) / (8 * kLanes<kF8>);
  const size_t n = blockIdx.x;
  const T* x = static_cast<const T*>(c.X) + n * c.ldx;
  const R* res = static_cast<const R*>(c.residual) + n * c.ldr;
  R* hout = static_cast<R*>(c.h) + n * c.ldh;
  float squares = 0.0f;
  for (int k0 = warp * 256; k0 < K; k0 += blockDim.x * 8) {
    const int k = k0 + 8 * lane;
    float v[8] = {};
    if (k < K) {
      float w[8];
      load8(x + k, v);
      load8_of(c.weight, c.wtype, k, w);
      if constexpr (kAdd) {
        float r[8];
        load8(res + k, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
        store8(hout + k, v);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        squares = fmaf(v[i], v[i], squares);
        v[i] *= w[i];
      }
    }
    const float top = group_max<kLanes<kF8>>(largest8(v));
    float sum = 0.0f;
    if (k < K) sum = store_codes<kF8>(o, n * K + k, v, top);
    if (!kF8 && o.us) {
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    }
    if (k < K && lane % kLanes<kF8> == 0) {
      const int b = k / (8 * kLanes<kF8>);
      kept[b] = top;
      if (!kF8 && o.us) kept[blocks + b] = sum;
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
    const float d = root * block_scale<kF8>(kept[b]);
    o.scale[(size_t)b * o.lds + n] = d;
    if (!kF8 && o.us) store_us(o.us, (int)n, K, b, d * kept[blocks + b]);
  }
}

// One block of 128 x 128 a CTA: a warp takes two rows at a time.
template <typename T>
__global__ void __launch_bounds__(256) weights_kernel(const T* W, int M, int K, long long ldw,
                                                      uint8_t* wq, float* sw) {
  __shared__ float tops[8];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int across = (K + kF8Block - 1) / kF8Block;
  const int mb = blockIdx.x / across, kb = blockIdx.x - mb * across;
  const int k = kb * kF8Block + 8 * (lane & 15);
  const long long m0 = (long long)mb * kF8Block + 2 * warp + (lane >> 4);
  float v[8][8] = {};
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const long long m = m0 + 16 * i;
    if (m < M && k < K) load8(W + m * ldw + k, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_nan(top, largest8(v[i]));
  top = group_max<32>(top);
  if (lane == 0) tops[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_nan(top, tops[i]);
  RowSink o = {};
  o.q = wq;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const long long m = m0 + 16 * i;
    if (m < M && k < K) store_codes<true>(o, (size_t)m * K + k, v[i], top);
  }
  if (threadIdx.x == 0) sw[blockIdx.x] = block_scale<true>(top);
}

template <typename T, bool kGlu>
cudaError_t rows_t(const void* X, int N, int K, long long ldx, const RowSink& out, cudaStream_t s) {
  const long long parts = (long long)N * ((K + 255) / 256);
  const long long blocks = (parts + 7) / 8;
  const unsigned grid = (unsigned)(blocks < 152 * 32 ? blocks : 152 * 32);
  return launch_pdl(out.f8 ? rows_kernel<T, true, kGlu> : rows_kernel<T, false, kGlu>, dim3(grid),
                    dim3(256), 0, s, static_cast<const T*>(X), N, K, ldx, out);
}
template <bool kGlu>
cudaError_t rows_of(const void* X, int type, int N, int K, long long ldx, const RowSink& out,
                    cudaStream_t s) {
  return type == Q6_TYPE_F32    ? rows_t<float, kGlu>(X, N, K, ldx, out, s)
         : type == Q6_TYPE_BF16 ? rows_t<__nv_bfloat16, kGlu>(X, N, K, ldx, out, s)
                                : rows_t<__half, kGlu>(X, N, K, ldx, out, s);
}

template <typename T, typename R, bool kAdd>
cudaError_t norm_t(const NormCall& c, const RowSink& out, cudaStream_t s) {
  int threads = (c.K + 255) / 256 * 32;
  if (threads > 1024) threads = 1024;
  const int blocks = (c.K + (out.f8 ? kF8Block : kQ8Block) - 1) / (out.f8 ? kF8Block : kQ8Block);
  const size_t smem = (size_t)blocks * (out.us ? 8 : 4);
  return launch_pdl(out.f8 ? norm_kernel<T, R, true, kAdd> : norm_kernel<T, R, false, kAdd>,
                    dim3((unsigned)c.N), dim3((unsigned)threads), smem, s, c, out);
}
template <typename T>
cudaError_t norm_of(const NormCall& c, const RowSink& out, cudaStream_t s) {
  if (!c.residual) return norm_t<T, T, false>(c, out, s);
  return c.rtype == Q6_TYPE_F32    ? norm_t<T, float, true>(c, out, s)
         : c.rtype == Q6_TYPE_BF16 ? norm_t<T, __nv_bfloat16, true>(c, out, s)
                                   : norm_t<T, __half, true>(c, out, s);
}
template <typename T>
cudaError_t weights_t(const void* W, int M, int K, long long ldw, uint8_t* wq, float* sw,
                      cudaStream_t s) {
  return launch_pdl(weights_kernel<T>, dim3((unsigned)f8_blocks(M) * (unsigned)f8_blocks(K)),
                    dim3(256), 0, s, static_cast<const T*>(W), M, K, ldw, wq, sw);
}

}  // namespace

cudaError_t launch_quantize_rows(const void* X, int type, int N, int K, long long ldx,
                                 const RowSink& out, cudaStream_t s) {
  return rows_of<false>(X, type, N, K, ldx, out, s);
}
cudaError_t launch_silu_mul(const void* X, int type, int N, int K, long long ldx,
                            const RowSink& out, cudaStream_t s) {
  return rows_of<true>(X, type, N, K, ldx, out, s);
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
