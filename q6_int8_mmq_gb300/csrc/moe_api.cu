// C-ABI entry points of the projections whose weights each token chooses:
// argument checks and kernel dispatch.
#include <cstdarg>

#include "moe_internal.cuh"

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

// Sizes of a grouping.
int check_group(int N, int per_row, int groups) {
  if (N < 0 || per_row < 1 || per_row > Q6_MAX_TOPK || groups < 1 || groups > Q6_MAX_GROUPS)
    return fail(Q6_EINVAL, "N >= 0, 1 <= items of a token <= %d, 1 <= groups <= %d", Q6_MAX_TOPK,
                Q6_MAX_GROUPS);
  if ((long long)N * per_row >= 1ll << 31) return fail(Q6_EINVAL, "N * per_row must be below 2^31");
  return Q6_OK;
}
size_t group_bytes(int N, int per_row, int groups) {
  const int blocks = q6::group_blocks((long long)N * per_row, N);
  return blocks > 1 ? (size_t)blocks * (size_t)q6::group_hist_ld(groups) * 4 : 0;
}
int check_group_buffers(const void* offsets, const void* rows, const void* pos, const void* ws,
                        size_t ws_bytes, size_t need, int N) {
  if (!offsets || (N > 0 && (!rows || !pos))) return fail(Q6_EINVAL, "null pointer");
  if (!aligned(offsets, 4) || !aligned(rows, 4) || !aligned(pos, 4) || !aligned(ws, 16))
    return fail(Q6_EALIGN, "offsets, rows and pos must be 4-byte, the workspace 16-byte aligned");
  if (need && (!ws || ws_bytes < need))
    return fail(Q6_ESIZE, "the grouping needs a workspace of %zu bytes", need);
  return Q6_OK;
}

int check_experts(int fmt, int E, int M, int K, int swiglu) {
  if (fmt != Q6_FMT_Q4K && fmt != Q6_FMT_Q6K) return fail(Q6_EINVAL, "unknown weight format %d", fmt);
  if (E < 1 || E > Q6_MAX_GROUPS || M < 1 || K < 1 || K % 256 || (swiglu && M % 2))
    return fail(Q6_EINVAL, "1 <= E <= %d, M >= 1 (even with swiglu), K a multiple of 256",
                Q6_MAX_GROUPS);
  if (q6::expert_rows(M, swiglu) > q6::kMaxPlaneRows)
    return fail(Q6_ESIZE, "an expert has more than %lld rows", q6::kMaxPlaneRows);
  const q6::ExpertGeom g = q6::expert_geom(fmt, E, M, K, swiglu);
  if ((long long)E * g.bands * (long long)g.sbs >= 1ll << 31)
    return fail(Q6_ESIZE, "the experts have too many tiles");
  return Q6_OK;
}

// The few-token kernel runs up to one item an expert on average. Measured, few-token
// kernel / tensor cores in us, with 0.5, 1, 2 and 4 items an expert: q4_K, 64 experts
// of 1536 x 2048 13.6 / 17.8, 24.2 / 24.2, 30.6 / 28.1, 46.6 / 30.4; 8 of 4096 x 4096
// 13.5 / 16.2, 22.7 / 23.5, 24.5 / 26.9, 33.6 / 27.0; q6_K, 32 of 2056 x 1536
// 13.4 / 15.0, 16.9 / 20.0, 24.3 / 23.8, 35.1 / 27.4.
bool on_tensor_cores(int64_t items, int E) { return items > E; }
// Bytes of the binary16 rows in item order that the tensor-core path makes (0:
// it reads X itself), and where their scales follow.
size_t rows_bytes(int64_t items, int K) { return q6::round_up((size_t)items * (size_t)K * 2, 256); }
size_t experts_bytes(int64_t items, int E, int K, int type, int gather) {
  if (!on_tensor_cores(items, E) || (type == Q6_TYPE_F16 && !gather)) return 0;
  return rows_bytes(items, K) + (type == Q6_TYPE_BF16 ? (size_t)items * 4 : 0);
}

bool half_type(int type) { return type == Q6_TYPE_BF16 || type == Q6_TYPE_F16; }
bool any_type(int type) { return half_type(type) || type == Q6_TYPE_F32; }

}  // namespace

extern "C" {

int q6_group_workspace_bytes(int N, int per_row, int groups, size_t* bytes) {
  const int rc = check_group(N, per_row, groups);
  if (rc) return rc;
  if (!bytes) return fail(Q6_EINVAL, "null pointer");
  *bytes = group_bytes(N, per_row, groups);
  return Q6_OK;
}

int q6_group_rows(const int32_t* ids, int N, int per_row, int groups, int32_t* offsets,
                  int32_t* rows, int32_t* pos, void* workspace, size_t workspace_bytes,
                  q6_stream_t s) {
  int rc = check_group(N, per_row, groups);
  if (rc) return rc;
  if (N > 0 && !ids) return fail(Q6_EINVAL, "null pointer");
  if (!aligned(ids, 4)) return fail(Q6_EALIGN, "ids must be 4-byte aligned");
  if ((rc = check_group_buffers(offsets, rows, pos, workspace, workspace_bytes,
                                group_bytes(N, per_row, groups), N)) ||
      (rc = q6::require_device(nullptr)))
    return rc;
  return launched(q6::launch_group(ids, N, per_row, groups, offsets, rows, pos,
                                   static_cast<int32_t*>(workspace), (cudaStream_t)s),
                  "grouping");
}

int q6_moe_route(const void* logits, int type, int N, int E, int64_t ldl, int topk,
                 int renormalize, int32_t* ids, float* weights, int32_t* offsets, int32_t* rows,
                 int32_t* pos, void* workspace, size_t workspace_bytes, q6_stream_t s) {
  int rc = check_group(N, topk, E);
  if (rc) return rc;
  if (!any_type(type)) return fail(Q6_EINVAL, "unknown type %d", type);
  if (topk > E || ldl < E) return fail(Q6_EINVAL, "topk <= E and ldl >= E");
  if (N > 0 && (!logits || !ids || !weights)) return fail(Q6_EINVAL, "null pointer");
  if (!aligned(logits, type == Q6_TYPE_F32 ? 4 : 2) || !aligned(ids, 4) || !aligned(weights, 4))
    return fail(Q6_EALIGN, "logits, ids and weights must be aligned to their elements");
  if ((rc = check_group_buffers(offsets, rows, pos, workspace, workspace_bytes,
                                group_bytes(N, topk, E), N)) ||
      (rc = q6::require_device(nullptr)))
    return rc;
  return launched(q6::launch_route(logits, type, N, E, ldl, topk, renormalize, ids, weights,
                                   offsets, rows, pos, static_cast<int32_t*>(workspace),
                                   (cudaStream_t)s),
                  "routing");
}

int q6_expert_plane_bytes(int fmt, int E, int M, int K, int swiglu, size_t* bytes) {
  const int rc = check_experts(fmt, E, M, K, swiglu);
  if (rc) return rc;
  if (!bytes) return fail(Q6_EINVAL, "null pointer");
  *bytes = q6::expert_geom(fmt, E, M, K, swiglu).total;
  return Q6_OK;
}

int q6_pack_experts(int fmt, const uint8_t* raw, int E, int M, int K, int swiglu, void* plane,
                    q6_stream_t s) {
  int rc = check_experts(fmt, E, M, K, swiglu);
  if (rc) return rc;
  if (!raw || !plane) return fail(Q6_EINVAL, "null pointer");
  if (!aligned(plane, 256)) return fail(Q6_EALIGN, "plane must be 256-byte aligned");
  const uint8_t* src;
  if ((rc = q6::require_device(nullptr)) || (rc = q6::readable_raw(raw, &src))) return rc;
  return launched(q6::launch_expert_pack(fmt, src, E, M, K, swiglu, static_cast<uint8_t*>(plane),
                                         (cudaStream_t)s),
                  "expert pack");
}

int q6_experts_workspace_bytes(int E, int K, int type, int64_t items, int gather, size_t* bytes) {
  if (E < 1 || K < 1 || K % 256 || !half_type(type) || items < 0 || items >= 1ll << 31 || !bytes)
    return fail(Q6_EINVAL,
                "E >= 1, K a multiple of 256, type bf16 or f16, 0 <= items < 2^31, bytes not NULL");
  *bytes = experts_bytes(items, E, K, type, gather);
  return Q6_OK;
}

int q6_experts_mmq(int fmt, const void* plane, int E, int M, int K, int swiglu, const void* X,
                   int type, int64_t nx, int64_t ldx, int gather, const int32_t* offsets,
                   const int32_t* rows, int64_t items, void* Y, int64_t ldy, void* workspace,
                   size_t workspace_bytes, int* path_out, q6_stream_t s) {
  int rc = check_experts(fmt, E, M, K, swiglu);
  if (rc) return rc;
  if (path_out) *path_out = Q6_PATH_NONE;
  q6::ExpertCall c;
  c.g = q6::expert_geom(fmt, E, M, K, swiglu);
  if (!half_type(type)) return fail(Q6_EINVAL, "X and Y must be bf16 or f16");
  if (items < 0 || items >= 1ll << 31 || nx < 0 || ldx < K || ldy < c.g.out)
    return fail(Q6_EINVAL, "0 <= items < 2^31, ldx >= K, ldy >= %d", c.g.out);
  if (!gather && nx < items) return fail(Q6_EINVAL, "X has fewer rows than there are items");
  if (items == 0) return Q6_OK;
  if (!plane || !X || !offsets || (gather && !rows) || !Y || nx == 0)
    return fail(Q6_EINVAL, "null pointer");
  if (!aligned(plane, 256) || !aligned(X, 16) || ldx % 8 || !aligned(Y, 2) || !aligned(offsets, 4) ||
      !aligned(rows, 4))
    return fail(Q6_EALIGN, "plane must be 256-byte, X and its rows 16-byte aligned");
  unsigned int* status;
  if ((rc = q6::require_device(&status, q6::kExpertKernels))) return rc;
  c.fmt = fmt, c.swiglu = swiglu, c.E = E;
  c.plane = static_cast<const uint8_t*>(plane);
  c.X = X, c.type = type, c.ldx = ldx, c.gather = gather;
  c.offsets = offsets, c.rows = rows, c.items = items;
  c.Y = Y, c.ldy = ldy;
  if (on_tensor_cores(items, E)) {
    const size_t need = experts_bytes(items, E, K, type, gather);
    if (need && (!workspace || workspace_bytes < need))
      return fail(Q6_ESIZE, "the product needs a workspace of %zu bytes", need);
    if (need && !aligned(workspace, 256)) return fail(Q6_EALIGN, "workspace must be 256-byte aligned");
    __half* xh = static_cast<__half*>(workspace);
    float* scale = nullptr;
    if (type == Q6_TYPE_BF16)
      scale = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + rows_bytes(items, K));
    q6::RowMaps maps;
    if ((rc = need ? q6::encode_row_maps(&maps, xh, items, K, K)
                   : q6::encode_row_maps(&maps, X, nx, K, ldx)))
      return rc;
    if (need && (rc = launched(q6::launch_expert_rows(c, K, xh, scale, (cudaStream_t)s),
                               "expert rows")))
      return rc;
    if (path_out) *path_out = Q6_PATH_EXPERTS_TC;
    return launched(
        q6::launch_experts_tc(c, maps, scale, need > 0, status, (cudaStream_t)s),
        "grouped product");
  }
  if (path_out) *path_out = Q6_PATH_EXPERTS_FEW;
  return launched(q6::launch_experts_few(c, (cudaStream_t)s), "grouped product");
}

int q6_moe_combine(const void* Y, int type, int64_t ldy, const int32_t* pos, const float* weights,
                   int N, int topk, int M, const float* shared, int64_t lds, void* out,
                   int64_t ldo, q6_stream_t s) {
  if (!half_type(type)) return fail(Q6_EINVAL, "Y and out must be bf16 or f16");
  if (N < 0 || topk < 1 || topk > Q6_MAX_TOPK || M < 1 || ldy < M || ldo < M || (shared && lds < M))
    return fail(Q6_EINVAL, "N >= 0, 1 <= topk <= %d, M >= 1 and leading dimensions >= M",
                Q6_MAX_TOPK);
  if (N == 0) return Q6_OK;
  if (!Y || !pos || !weights || !out) return fail(Q6_EINVAL, "null pointer");
  if (!aligned(Y, 2) || !aligned(out, 2) || !aligned(pos, 4) || !aligned(weights, 4) ||
      !aligned(shared, 4))
    return fail(Q6_EALIGN, "a pointer is not aligned to its elements");
  const int rc = q6::require_device(nullptr);
  if (rc) return rc;
  return launched(q6::launch_combine(Y, type, ldy, pos, weights, N, topk, M, shared, lds, out, ldo,
                                     (cudaStream_t)s),
                  "combination");
}

// Widths and items up to which the adapters' kernels' indices, which run up to a
// step past the end, stay within 31 bits.
static constexpr int kLoraMaxWidth = 1 << 30;
static constexpr int64_t kLoraMaxItems = (1ll << 31) - 256;

static int check_lora(int64_t items, int L, int r, int K) {
  if (items < 0 || items >= 1ll << 31 || L < 1 || L > Q6_MAX_GROUPS)
    return fail(Q6_EINVAL, "0 <= items < 2^31, 1 <= L <= %d", Q6_MAX_GROUPS);
  if (items > kLoraMaxItems || K > kLoraMaxWidth)
    return fail(Q6_ESIZE, "more than 2^31 - 256 items, or K above 2^30");
  if (r < 8 || r % 8 || r > Q6_LORA_MAX_RANK || K < 32 || K % 32)
    return fail(Q6_EINVAL, "the rank must be a multiple of 8 up to %d (pad with zeros), K one of 32",
                Q6_LORA_MAX_RANK);
  return Q6_OK;
}

int q6_lora_workspace_bytes(int64_t items, int L, int r, int K, size_t* bytes) {
  const int rc = check_lora(items, L, r, K);
  if (rc) return rc;
  if (!bytes) return fail(Q6_EINVAL, "null pointer");
  *bytes = (size_t)q6::lora_splits(items, L, r, K) * (size_t)items * (size_t)r * 4;
  return Q6_OK;
}

int q6_lora_add(const void* A, const void* B, const float* scale, int type, int L, int r, int M,
                int K, const void* X, int xtype, int64_t ldx, const int32_t* offsets,
                const int32_t* rows, int64_t items, const float* Y, int64_t ldy, float* out,
                int64_t ldo, void* workspace, size_t workspace_bytes, q6_stream_t s) {
  int rc = check_lora(items, L, r, K);
  if (rc) return rc;
  if (!half_type(type) || !any_type(xtype))
    return fail(Q6_EINVAL, "adapters must be bf16 or f16, X f32, bf16 or f16");
  if (M < 1 || ldx < K || ldy < M || ldo < M)
    return fail(Q6_EINVAL, "M >= 1, ldx >= K, ldy >= M, ldo >= M");
  if (M > kLoraMaxWidth) return fail(Q6_ESIZE, "M above 2^30");
  if (items == 0) return Q6_OK;
  if (!A || !B || !scale || !X || !offsets || !rows || !Y || !out)
    return fail(Q6_EINVAL, "null pointer");
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(X, 16) ||
      ldx * (xtype == Q6_TYPE_F32 ? 4 : 2) % 16 || !aligned(workspace, 16))
    return fail(Q6_EALIGN, "A, B, the rows of X and the workspace must be 16-byte aligned");
  if (!aligned(Y, 4) || !aligned(out, 4) || !aligned(scale, 4) || !aligned(offsets, 4) ||
      !aligned(rows, 4))
    return fail(Q6_EALIGN, "a pointer is not aligned to its elements");
  q6::LoraCall c;
  c.splits = q6::lora_splits(items, L, r, K);
  const size_t need = (size_t)c.splits * (size_t)items * (size_t)r * 4;
  if (need && (!workspace || workspace_bytes < need))
    return fail(Q6_ESIZE, "the adapters need a workspace of %zu bytes", need);
  if ((rc = q6::require_device(nullptr, q6::kAdapterKernels))) return rc;
  c.A = A, c.B = B, c.scale = scale, c.type = type;
  c.L = L, c.r = r, c.K = K, c.M = M;
  c.X = X, c.xtype = xtype, c.ldx = ldx;
  c.offsets = offsets, c.rows = rows, c.items = items;
  c.Y = Y, c.ldy = ldy, c.out = out, c.ldo = ldo;
  c.part = static_cast<float*>(workspace);
  return launched(q6::launch_lora(c, (cudaStream_t)s), "adapter");
}

}  // extern "C"
