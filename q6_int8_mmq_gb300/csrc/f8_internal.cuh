// Internal declarations of the 8-bit steps around the projections: activations
// quantised by the norm or the gated activation that makes them, and the
// products of e4m3 blocks.
#pragma once

#include "moe_internal.cuh"

namespace q6 {

// Elements of one scale: of a row of int8 codes, and of a row (or a side of a
// weight block) of e4m3 codes.
constexpr int kQ8Block = 32, kF8Block = 128;
inline int f8_blocks(int n) { return (int)(((long long)n + kF8Block - 1) / kF8Block); }
// Distance of the scale rows: N rounded up to 4.
inline int scale_ld(int N) { return (int)(((long long)N + 3) / 4 * 4); }

// Where quantised rows go: int8 (q, xh, us as q8_quantize_act_sums; any of them
// NULL) or e4m3 (q), with their scales [blocks][lds].
struct RowSink {
  bool f8;
  uint8_t* q;
  __half* xh;
  float* us;
  float* scale;
  int lds;
};
// Rows of X [N][ldx] as e4m3 codes.
cudaError_t launch_f8_quantize_rows(const void* X, int type, int N, int K, long long ldx,
                                    const RowSink& out, cudaStream_t s);
// silu(gate) * up of rows [N][ldx] of K gate, then K up values.
cudaError_t launch_silu_mul(const void* X, int type, int N, int K, long long ldx,
                            const RowSink& out, cudaStream_t s);
struct NormCall {
  const void* X;
  int type;
  long long ldx;
  const void* residual;  // or NULL
  int rtype;
  long long ldr;
  const void* weight;
  int wtype;
  float eps;
  int N, K;
  void* h;  // of rtype; NULL without residual
  long long ldh;
};
cudaError_t launch_rms_norm(const NormCall& c, const RowSink& out, cudaStream_t s);
cudaError_t launch_f8_quantize_weights(const void* W, int type, int M, int K, long long ldw,
                                       uint8_t* wq, float* sw, cudaStream_t s);

struct F8Call {
  const uint8_t* wq;
  const float* sw;
  int M, K;
  const uint8_t* xq;
  const float* sx;
  int N, ldsx;
  void* Y;
  int type;
  long long ldy;
};
// A tensor map of bytes [rows][K] in boxes of 128 of K x `box` rows with the
// 128-byte swizzle (api.cu).
int encode_f8_map(CUtensorMap* map, const void* base, int rows, int K, int box, const char* what);
// Token scales [rows][ld] in boxes of n tokens x `box` rows.
int encode_f8_scales(CUtensorMap* map, const float* sx, int ld, int rows, int n, int box);
// Y in boxes of `cols` x `rows` with the 64-byte swizzle.
int encode_f8_results(CUtensorMap* map, const F8Call& c, int cols, int rows);
// How a product of these sizes runs on the current device (prepared): a tile's tokens and
// weight rows, the parts of K that the CTAs (or pairs of CTAs) of a cluster take, and the
// clusters of that many that run at a time (0 where the device could not say).
struct F8Form {
  int tokens, rows, parts, room;
};
cudaError_t f8_few_form(int M, int K, int N, F8Form* form);
cudaError_t f8_tc_form(int M, int K, int N, F8Form* form);
// *e receives the launch's error; returns Q6_OK, or a code whose text is recorded.
cudaError_t f8_few_prepare();
int launch_f8_few(const F8Call& c, cudaError_t* e, unsigned int* status, cudaStream_t s);
cudaError_t f8_tc_prepare();
int launch_f8_tc(const F8Call& c, cudaError_t* e, unsigned int* status, cudaStream_t s);

}  // namespace q6
