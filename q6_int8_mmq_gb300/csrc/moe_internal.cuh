// Internal declarations of the per-token weight choice: expert routing and
// grouping, the grouped products of K-quant experts, their combination, and
// low-rank adapters.
#pragma once

#include <cuda_bf16.h>

#include "q6_internal.cuh"

namespace q6 {

// Kernels that have attributes to raise before their first launch. That loads them
// (1.7 ms for the two sets together, 2.1 ms for the kernels of the shared projections),
// so each set is prepared by the first call that runs it.
enum KernelSet { kPlainKernels, kExpertKernels, kAdapterKernels, kBlockKernels, kKernelSets };
constexpr int kMaxDevices = 64;
// The calling thread's current device, checked and prepared, and `set` on it
// (api.cu); *status (nullable) receives its status word.
int require_device(unsigned int** status, KernelSet set = kPlainKernels);
// The address a kernel reads raw weight bytes through (api.cu).
int readable_raw(const uint8_t* raw, const uint8_t** src);

// ------------------------------------------------------- routing, grouping ---
constexpr int kMaxGroups = Q6_MAX_GROUPS;
// Blocks that share one grouping: each owns a contiguous range of rows. One
// block up to kGroupSingle items, else up to one an SM (8191 tokens to 8 of 256
// experts 16.1 us, with 128 blocks 17.2).
constexpr int kGroupBlocks = 152;
constexpr int kGroupSingle = 512;
inline int group_blocks(long long items, int N) {
  if (items <= kGroupSingle || N <= 1) return 1;
  return N < kGroupBlocks ? N : kGroupBlocks;
}
// Row length of the blocks' counts: groups and the section of none, padded.
__host__ __device__ constexpr int group_hist_ld(int G) { return (G + 4) / 4 * 4; }
cudaError_t launch_route(const void* logits, int type, int N, int E, long long ldl, int topk,
                         int renorm, int32_t* ids, float* weights, int32_t* offsets,
                         int32_t* rows, int32_t* pos, int32_t* hist, cudaStream_t s);
cudaError_t launch_group(const int32_t* ids, int N, int per_row, int G, int32_t* offsets,
                         int32_t* rows, int32_t* pos, int32_t* hist, cudaStream_t s);
cudaError_t launch_combine(const void* Y, int type, long long ldy, const int32_t* pos,
                           const float* weights, int N, int topk, int M, const float* shared,
                           long long lds, void* out, long long ldo, cudaStream_t s);

// ---------------------------------------------------------------- elements ---
template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Two 16-bit values of a word as f32, and the reverse (one rounding each).
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

}  // namespace q6

namespace q6 {

// binary16 pairs.
__device__ __forceinline__ uint32_t hmul2u(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hfma2u(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t word4(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// ------------------------------------------------------------ expert plane ---
// Packed K-quant experts: per expert and band of 128 plane rows, one tile per
// super-block (256 elements of K), tiles in the order [expert][band][super-
// block], each contiguous, so a kernel streams its weights front to back.
// Inside a tile everything is split into 16-byte units laid out [unit][row]:
// 128 consecutive threads that take one row each, or 8 rows x 4 lanes of an
// MMA fragment, read whole 128-byte lines.
//
// The 256 elements of a row are 8 chunks c of 32, a chunk 4 runs t of 8. A
// 32-bit nibble word holds one run: element 2m in nibble m, element 2m + 1 in
// nibble m + 4, so (word >> 4m) & 0x000F000F is the pair (2m, 2m + 1) as the
// two halves of a register. Unit j = 2t + h holds the words of run t of
// chunks 4h..4h+3.
//   q4_K (9 units): 0: d, dmin (f16) and the 12 raw scale bytes; 1 + j: words.
//   q6_K (13 units and 256 bytes): j: low-nibble words; 8 + t: the 2-bit
//     fields of run t, word c/2, pair m at bit 4 m + 2 (c % 2) of each half;
//     12: the 16 scales plus 128, those of even sub-blocks first; then d (f16)
//     of the 128 rows.
// After the tiles, f32 [E][bands * 128]: 2^e of each row, with e such that
// every weight of the row times 2^-e is below 2^10; -2^e for 32 rows of which one
// has super-blocks far smaller than its largest. As binary16 at that size a weight is
// rounded to 11 bits, or by at most 2^-34 of the row's largest possible one; bf16
// products of other rows take it 2^15 smaller, by at most 2^-19 (experts_tc.cu).
//
// Plane rows: the weight's rows, or for gate/up weights (M = 2H raw rows, the
// H gate rows first) blocks of 16: 8 gate rows, then their 8 up rows.
constexpr int kBand = 128;
constexpr int kQ4Tile = 9 * 2048;
constexpr int kQ6Tile = 13 * 2048 + 256;

// The 6-bit codes of a run of a q6_K chunk (c % 2 = odd), pairs in halves:
// word w of low nibbles, word h of 2-bit fields.
__device__ __forceinline__ void q6_pairs(uint32_t w, uint32_t h, int odd, uint32_t (&v)[4]) {
  // nibbles 0 and 2 with their fields above them, then 1 and 3
  const uint32_t even = (w & 0x0F0F0F0Fu) | ((h << (odd ? 2 : 4)) & ~0x0F0F0F0Fu);
  const uint32_t rest = ((w >> 4) & 0x0F0F0F0Fu) | ((odd ? h >> 2 : h) & ~0x0F0F0F0Fu);
  v[0] = even & 0x003F003Fu;
  v[1] = rest & 0x003F003Fu;
  v[2] = (even >> 8) & 0x003F003Fu;
  v[3] = (rest >> 8) & 0x003F003Fu;
}

struct ExpertGeom {
  int rows;        // plane rows
  int bands;       // per expert
  int sbs;         // super-blocks of K
  int tile;        // bytes
  int out;         // output features: M, or M / 2 with swiglu
  size_t scale_off, total;
};
// Plane rows of an expert (up to 2^31 + 8), and the most that leave the kernels'
// row numbers, which run up to 128 + 32 past the last row, within 31 bits.
constexpr long long kMaxPlaneRows = (1ll << 31) - 256;
inline long long expert_rows(int M, int swiglu) {
  return swiglu ? (M / 2 + 7ll) / 8 * 16 : M;
}
inline ExpertGeom expert_geom(int fmt, int E, int M, int K, int swiglu) {
  ExpertGeom g;
  g.out = swiglu ? M / 2 : M;
  g.rows = (int)expert_rows(M, swiglu);
  g.bands = (g.rows + kBand - 1) / kBand;
  g.sbs = K / 256;
  g.tile = fmt == Q6_FMT_Q4K ? kQ4Tile : kQ6Tile;
  g.scale_off = (size_t)E * (size_t)g.bands * (size_t)g.sbs * (size_t)g.tile;
  g.total = g.scale_off + (size_t)E * (size_t)g.bands * kBand * 4;
  return g;
}

cudaError_t launch_expert_pack(int fmt, const uint8_t* raw, int E, int M, int K, int swiglu,
                               uint8_t* plane, cudaStream_t s);

// One grouped product (see q6_experts_mmq).
struct ExpertCall {
  int fmt, swiglu, E;
  ExpertGeom g;
  const uint8_t* plane;
  const void* X;
  int type;           // of X and Y
  long long ldx;      // of X rows
  int gather;         // X row of item i: rows[i], else i
  const int32_t* offsets;
  const int32_t* rows;
  long long items;
  void* Y;
  long long ldy;
};
cudaError_t experts_few_prepare();
cudaError_t launch_experts_few(const ExpertCall& c, cudaStream_t s);
cudaError_t experts_tc_prepare();
// Tensor maps of binary16 rows [n][ld] as boxes of 64 elements x 16, 32, 64 and
// 128 rows with the 128-byte swizzle.
struct RowMaps {
  static constexpr int kCount = 4;
  CUtensorMap box[kCount];
};
int encode_row_maps(RowMaps* maps, const void* X, long long n, int K, long long ld);
// x: the items' rows as binary16 in order, scale (nullable): f32 [items], what
// each is multiplied with; x_made: launch_expert_rows has just made them on s.
// c.X, c.gather and c.rows are not used.
cudaError_t launch_experts_tc(const ExpertCall& c, const RowMaps& x, const float* scale,
                              bool x_made, unsigned int* status, cudaStream_t s);
// The items' rows of X as binary16 in item order: xh [items][K], and for bf16
// (scaled by a power of two of the row) scale [items], that power.
cudaError_t launch_expert_rows(const ExpertCall& c, int K, __half* xh, float* scale,
                               cudaStream_t s);

}  // namespace q6

namespace q6 {

// ----------------------------------------------------------------- adapters ---
struct LoraCall {
  const void* A;  // [L][r][K]
  const void* B;  // [L][M][r]
  const float* scale;
  int type;       // of A and B
  int L, r, K, M;
  const void* X;
  int xtype;
  long long ldx;
  const int32_t* offsets;
  const int32_t* rows;
  long long items;
  const float* Y;
  long long ldy;
  float* out;
  long long ldo;
  float* part;    // K-part sums [splits][items][r]
  int splits;
};
// Parts the shrink product splits K into (its workspace is splits * items * r
// f32 values); 0 where one kernel does it all.
int lora_splits(long long items, int L, int r, int K);
cudaError_t lora_prepare();
cudaError_t launch_lora(const LoraCall& c, cudaStream_t s);

}  // namespace q6
