// C-ABI entry points of the 8-bit steps around the projections: argument checks
// and kernel dispatch.
#include <cstdarg>
#include <cfloat>

#include "f8_internal.cuh"

namespace q6 {
int record_error(int code, const char* fmt, va_list ap);  // defined with q6_last_error()
}

namespace {

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  const int rc = q6::record_error(code, fmt, ap);
  va_end(ap);
  return rc;
}

int launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? Q6_OK : fail(Q6_ECUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool any_type(int type) {
  return type == Q6_TYPE_F32 || type == Q6_TYPE_BF16 || type == Q6_TYPE_F16;
}
// Rows of `type` that start on 16 bytes (ld: elements).
bool rows_aligned(const void* p, int type, int64_t ld) {
  return aligned(p, 16) && ld % (type == Q6_TYPE_F32 ? 4 : 8) == 0;
}

// Sizes up to which the kernels' indices, which run up to four parts of 512 past the
// end, stay within 31 bits.
constexpr int kMost = INT32_MAX - 4096;
constexpr int64_t kMostElements = 1ll << 40;

// Tokens up to which the weight's rows are the tensor cores' lanes. (The next width, 128
// tokens that way, eight warps summing: 11008 x 4096 23.9 us, 4096 x 4096 15.8 and 4096 x
// 11008 25.4; tokens on the lanes 18.0, 10.5 and 18.1. 64 tokens this way 12.8, 8.2 and
// 12.8, 65 the other way 17.6, 10.2 and 17.8.)
constexpr int kFewTokens = 64;

int check_f8(int rows, int K) {
  if (rows < 0 || K < 1 || K % 16) return fail(Q6_EINVAL, "rows >= 0, K a positive multiple of 16");
  if (rows > kMost || K > kMost || (int64_t)rows * K > kMostElements)
    return fail(Q6_ESIZE, "more than %d rows or columns, or 2^40 elements", kMost);
  return Q6_OK;
}
int check_q8(int N, int K) {
  if (N < 0 || K < 1 || K % 256) return fail(Q6_EINVAL, "N >= 0, K a positive multiple of 256");
  return check_f8(N, K);
}
int check_q8_sink(const int8_t* Xq, const float* da, const uint16_t* Xh, const float* us) {
  if (!da || (!Xq && !Xh)) return fail(Q6_EINVAL, "da and one of Xq, Xh are required");
  if (!aligned(Xq, 16) || !aligned(da, 16) || !aligned(Xh, 16) || !aligned(us, 16))
    return fail(Q6_EALIGN, "Xq, da, Xh and us must be 16-byte aligned");
  return Q6_OK;
}
int check_f8_sink(const uint8_t* xq, const float* sx) {
  if (!xq || !sx) return fail(Q6_EINVAL, "null pointer");
  if (!aligned(xq, 16) || !aligned(sx, 16)) return fail(Q6_EALIGN, "xq and sx must be 16-byte aligned");
  return Q6_OK;
}
q6::RowSink q8_sink(int N, int8_t* Xq, float* da, uint16_t* Xh, float* us) {
  return {false, reinterpret_cast<uint8_t*>(Xq), reinterpret_cast<__half*>(Xh), us, da,
          q6::scale_ld(N)};
}
q6::RowSink f8_sink(int N, uint8_t* xq, float* sx) {
  return {true, xq, nullptr, nullptr, sx, q6::scale_ld(N)};
}

int check_rows(const void* X, int type, int64_t ldx, int64_t width) {
  if (!any_type(type)) return fail(Q6_EINVAL, "unknown type %d", type);
  if (ldx < width) return fail(Q6_EINVAL, "ldx (%lld) is below the rows' width", (long long)ldx);
  if (!X) return fail(Q6_EINVAL, "null pointer");
  if (!rows_aligned(X, type, ldx)) return fail(Q6_EALIGN, "rows must be 16-byte aligned");
  return Q6_OK;
}

int check_product(int M, int K, int N) {
  int rc = check_f8(N, K);
  if (rc || (rc = check_f8(M, K))) return rc;
  if (M < 1) return fail(Q6_EINVAL, "M >= 1");
  // blocks of all tiles, which a CTA may have to count
  if ((double)q6::f8_blocks(M) * q6::f8_blocks(N) * q6::f8_blocks(K) > INT32_MAX)
    return fail(Q6_ESIZE, "the product has too many tiles");
  return Q6_OK;
}

int norm_entry(const q6::NormCall& c, const q6::RowSink& out, q6_stream_t s) {
  if (!any_type(c.type) || !any_type(c.wtype) || (c.residual && !any_type(c.rtype)))
    return fail(Q6_EINVAL, "unknown type");
  if (!(c.eps >= FLT_MIN && c.eps <= FLT_MAX))
    return fail(Q6_EINVAL, "eps must be a positive normal number");
  if (c.K > Q6_NORM_MAX_K) return fail(Q6_ESIZE, "K above %d", Q6_NORM_MAX_K);
  int rc = check_rows(c.X, c.type, c.ldx, c.K);
  if (rc) return rc;
  if (!c.weight || (c.residual && !c.h)) return fail(Q6_EINVAL, "null pointer");
  if (!aligned(c.weight, 16)) return fail(Q6_EALIGN, "weight must be 16-byte aligned");
  if (c.residual) {
    if (c.ldr < c.K || c.ldh < c.K) return fail(Q6_EINVAL, "ldr >= K and ldh >= K");
    if (!rows_aligned(c.residual, c.rtype, c.ldr) || !rows_aligned(c.h, c.rtype, c.ldh))
      return fail(Q6_EALIGN, "rows must be 16-byte aligned");
  } else if (c.h) {
    return fail(Q6_EINVAL, "h without a residual");
  }
  if ((rc = q6::require_device(nullptr))) return rc;
  return launched(q6::launch_rms_norm(c, out, (cudaStream_t)s), "norm");
}

}  // namespace

extern "C" {

int q6_f8_act_bytes(int N, int K, size_t* xq_bytes, size_t* sx_bytes, int* ldsx) {
  const int rc = check_f8(N, K);
  if (rc) return rc;
  if (xq_bytes) *xq_bytes = (size_t)N * (size_t)K;
  if (sx_bytes) *sx_bytes = (size_t)q6::f8_blocks(K) * (size_t)q6::scale_ld(N) * 4;
  if (ldsx) *ldsx = q6::scale_ld(N);
  return Q6_OK;
}

int q6_f8_weight_bytes(int M, int K, size_t* wq_bytes, size_t* sw_bytes) {
  const int rc = check_f8(M, K);
  if (rc) return rc;
  if (M < 1) return fail(Q6_EINVAL, "M >= 1");
  if (wq_bytes) *wq_bytes = (size_t)M * (size_t)K;
  if (sw_bytes) *sw_bytes = (size_t)q6::f8_blocks(M) * (size_t)q6::f8_blocks(K) * 4;
  return Q6_OK;
}

int q6_f8_quantize_act(const void* X, int type, int N, int K, int64_t ldx, uint8_t* xq, float* sx,
                       q6_stream_t s) {
  int rc = check_f8(N, K);
  if (rc || N == 0) return rc;
  if ((rc = check_rows(X, type, ldx, K)) || (rc = check_f8_sink(xq, sx)) ||
      (rc = q6::require_device(nullptr)))
    return rc;
  return launched(q6::launch_f8_quantize_rows(X, type, N, K, ldx, f8_sink(N, xq, sx),
                                              (cudaStream_t)s),
                  "quantiser");
}

int q6_f8_quantize_weights(const void* W, int type, int M, int K, int64_t ldw, uint8_t* wq,
                           float* sw, q6_stream_t s) {
  int rc = check_f8(M, K);
  if (rc) return rc;
  if (M < 1) return fail(Q6_EINVAL, "M >= 1");
  if ((rc = check_rows(W, type, ldw, K))) return rc;
  if (!wq || !sw) return fail(Q6_EINVAL, "null pointer");
  if (!aligned(wq, 16) || !aligned(sw, 4))
    return fail(Q6_EALIGN, "wq must be 16-byte, sw 4-byte aligned");
  if ((rc = q6::require_device(nullptr))) return rc;
  return launched(q6::launch_f8_quantize_weights(W, type, M, K, ldw, wq, sw, (cudaStream_t)s),
                  "weight quantiser");
}

int q6_rms_norm_q8(const void* X, int type, int64_t ldx, const void* residual, int rtype,
                   int64_t ldr, const void* weight, int wtype, float eps, int N, int K, void* h,
                   int64_t ldh, int8_t* Xq, float* da, uint16_t* Xh, float* us, q6_stream_t s) {
  int rc = check_q8(N, K);
  if (rc || N == 0 || (rc = check_q8_sink(Xq, da, Xh, us))) return rc;
  return norm_entry({X, type, ldx, residual, rtype, ldr, weight, wtype, eps, N, K, h, ldh},
                    q8_sink(N, Xq, da, Xh, us), s);
}

int q6_rms_norm_f8(const void* X, int type, int64_t ldx, const void* residual, int rtype,
                   int64_t ldr, const void* weight, int wtype, float eps, int N, int K, void* h,
                   int64_t ldh, uint8_t* xq, float* sx, q6_stream_t s) {
  int rc = check_f8(N, K);
  if (rc || N == 0 || (rc = check_f8_sink(xq, sx))) return rc;
  return norm_entry({X, type, ldx, residual, rtype, ldr, weight, wtype, eps, N, K, h, ldh},
                    f8_sink(N, xq, sx), s);
}

int q6_silu_mul_q8(const void* X, int type, int N, int K, int64_t ldx, int8_t* Xq, float* da,
                   uint16_t* Xh, float* us, q6_stream_t s) {
  int rc = check_q8(N, K);
  if (rc || N == 0) return rc;
  if ((rc = check_rows(X, type, ldx, 2 * (int64_t)K)) || (rc = check_q8_sink(Xq, da, Xh, us)) ||
      (rc = q6::require_device(nullptr)))
    return rc;
  return launched(q6::launch_silu_mul(X, type, N, K, ldx, q8_sink(N, Xq, da, Xh, us),
                                      (cudaStream_t)s),
                  "gated activation");
}

int q6_silu_mul_f8(const void* X, int type, int N, int K, int64_t ldx, uint8_t* xq, float* sx,
                   q6_stream_t s) {
  int rc = check_f8(N, K);
  if (rc || N == 0) return rc;
  if ((rc = check_rows(X, type, ldx, 2 * (int64_t)K)) || (rc = check_f8_sink(xq, sx)) ||
      (rc = q6::require_device(nullptr)))
    return rc;
  return launched(q6::launch_silu_mul(X, type, N, K, ldx, f8_sink(N, xq, sx), (cudaStream_t)s),
                  "gated activation");
}

int q6_f8_mmq_form(int M, int K, int N, int* path, int* tokens, int* rows, int* parts, int* room) {
  if (!path || !tokens || !rows || !parts || !room) return fail(Q6_EINVAL, "null pointer");
  *path = Q6_PATH_NONE;
  *tokens = *rows = *parts = *room = 0;
  int rc = check_product(M, K, N);
  if (rc || N == 0 || (rc = q6::require_device(nullptr, q6::kBlockKernels))) return rc;
  const bool few = N <= kFewTokens;
  q6::F8Form f = {};
  const cudaError_t e = few ? q6::f8_few_form(M, K, N, &f) : q6::f8_tc_form(M, K, N, &f);
  if (e) return fail(Q6_ECUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  *path = few ? Q6_PATH_F8_FEW : Q6_PATH_F8_TC;
  *tokens = f.tokens, *rows = f.rows, *parts = f.parts, *room = f.room;
  return Q6_OK;
}

int q6_f8_mmq(const uint8_t* wq, const float* sw, int M, int K, const uint8_t* xq, const float* sx,
              int N, void* Y, int type, int64_t ldy, int* path_out, q6_stream_t s) {
  if (path_out) *path_out = Q6_PATH_NONE;
  int rc = check_product(M, K, N);
  if (rc) return rc;
  if (!any_type(type)) return fail(Q6_EINVAL, "unknown type %d", type);
  if (ldy < M) return fail(Q6_EINVAL, "ldy (%lld) < M (%d)", (long long)ldy, M);
  if (N == 0) return Q6_OK;
  if (!wq || !sw || !xq || !sx || !Y) return fail(Q6_EINVAL, "null pointer");
  if (!aligned(wq, 16) || !aligned(xq, 16) || !aligned(sx, 16) || !aligned(sw, 4) ||
      !aligned(Y, type == Q6_TYPE_F32 ? 4 : 2))
    return fail(Q6_EALIGN, "wq, xq and sx must be 16-byte aligned, sw and Y to their elements");
  unsigned int* status;
  if ((rc = q6::require_device(&status, q6::kBlockKernels))) return rc;
  const q6::F8Call c = {wq, sw, M, K, xq, sx, N, q6::scale_ld(N), Y, type, ldy};
  const bool few = N <= kFewTokens;
  cudaError_t e = cudaSuccess;
  if ((rc = few ? q6::launch_f8_few(c, &e, status, (cudaStream_t)s)
                : q6::launch_f8_tc(c, &e, status, (cudaStream_t)s)))
    return rc;
  if (path_out) *path_out = few ? Q6_PATH_F8_FEW : Q6_PATH_F8_TC;
  return launched(e, "block product");
}

}  // extern "C"
