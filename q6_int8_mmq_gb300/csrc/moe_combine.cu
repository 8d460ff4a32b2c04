// The combination of the experts' outputs:
//   out[n] = shared[n] + sum over slots j of weights[n][j] * Y[pos[n][j]],
// summed in f32 in slot order and rounded once to Y's type; a slot with pos
// < 0 adds nothing (its weight is not looked at).
//
// Bound: memory (every Y row is read once). A thread owns 8 columns of one
// token, so its slots' 16-byte loads are independent and in flight together: 4096
// tokens of 8 slots and 4096 bf16 columns with a shared f32 term take 51.2 us,
// 7.2 TB/s, a little above what a plain copy reaches.
#include "moe_internal.cuh"

namespace q6 {
namespace {

constexpr int kThreads = 128;

// kVec: rows of Y, out and shared are 16-byte aligned and M % 8 == 0.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
combine_kernel(const T* Y, long long ldy, const int32_t* pos, const float* weights, int topk,
               int M, const float* shared, long long lds, T* out, long long ldo) {
  griddep_wait();
  const size_t n = blockIdx.x;
  const int c0 = (blockIdx.y * kThreads + threadIdx.x) * (kVec ? 8 : 1);
  if (c0 >= M) return;
  const int32_t* p = pos + n * topk;
  const float* w = weights + n * topk;
  if constexpr (kVec) {
    float acc[8] = {};
    if (shared) {
      const float4 a = *reinterpret_cast<const float4*>(shared + n * lds + c0);
      const float4 b = *reinterpret_cast<const float4*>(shared + n * lds + c0 + 4);
      acc[0] = a.x, acc[1] = a.y, acc[2] = a.z, acc[3] = a.w;
      acc[4] = b.x, acc[5] = b.y, acc[6] = b.z, acc[7] = b.w;
    }
    for (int j0 = 0; j0 < topk; j0 += 8) {
      uint4 v[8];
      float wj[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = j0 + j < topk ? p[j0 + j] : -1;
        wj[j] = at >= 0 ? w[j0 + j] : 0.0f;
        v[j] = make_uint4(0, 0, 0, 0);
        if (at >= 0) v[j] = __ldcs(reinterpret_cast<const uint4*>(Y + (size_t)at * ldy + c0));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack2<T>(u[i]);
          acc[2 * i] = fmaf(wj[j], f.x, acc[2 * i]);
          acc[2 * i + 1] = fmaf(wj[j], f.y, acc[2 * i + 1]);
        }
      }
    }
    uint4 r;
    r.x = pack2<T>(acc[0], acc[1]);
    r.y = pack2<T>(acc[2], acc[3]);
    r.z = pack2<T>(acc[4], acc[5]);
    r.w = pack2<T>(acc[6], acc[7]);
    *reinterpret_cast<uint4*>(out + n * ldo + c0) = r;
  } else {
    float acc = shared ? shared[n * lds + c0] : 0.0f;
    for (int j = 0; j < topk; ++j)
      if (p[j] >= 0) acc = fmaf(w[j], to_f32(Y[(size_t)p[j] * ldy + c0]), acc);
    out[n * ldo + c0] = from_f32<T>(acc);
  }
}

bool aligned16(const void* p, long long ld_bytes) {
  return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)ld_bytes) % 16 == 0;
}

template <typename T>
cudaError_t combine_t(const void* Y, long long ldy, const int32_t* pos, const float* weights,
                      int N, int topk, int M, const float* shared, long long lds, void* out,
                      long long ldo, cudaStream_t s) {
  const bool vec = M % 8 == 0 && aligned16(Y, ldy * 2) && aligned16(out, ldo * 2) &&
                   (!shared || aligned16(shared, lds * 4));
  // a launch takes as many columns as a grid has blocks for (65535 of 128 or 1024)
  const int per = kThreads * (vec ? 8 : 1), most = 65535 * per;
  for (int m = 0;;) {
    const int cols = M - m < most ? M - m : most;
    const dim3 grid((unsigned)N, (unsigned)((cols + per - 1) / per));
    const cudaError_t e = launch_pdl(
        vec ? combine_kernel<T, true> : combine_kernel<T, false>, grid, dim3(kThreads), 0, s,
        static_cast<const T*>(Y) + m, ldy, pos, weights, topk, cols, shared ? shared + m : nullptr,
        lds, static_cast<T*>(out) + m, ldo);
    if (e != cudaSuccess || cols == M - m) return e;
    m += cols;
  }
}

}  // namespace

cudaError_t launch_combine(const void* Y, int type, long long ldy, const int32_t* pos,
                           const float* weights, int N, int topk, int M, const float* shared,
                           long long lds, void* out, long long ldo, cudaStream_t s) {
  return type == Q6_TYPE_BF16
             ? combine_t<__nv_bfloat16>(Y, ldy, pos, weights, N, topk, M, shared, lds, out, ldo, s)
             : combine_t<__half>(Y, ldy, pos, weights, N, topk, M, shared, lds, out, ldo, s);
}

}  // namespace q6
