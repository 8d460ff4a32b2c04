// Grouped K-quant expert products for few tokens an expert.
//
//   Y[i][m] = sum_k W[e(i)][m][k] x[t(i)][k],  W = d * sc * (q - 32)  (q6_K)
//                                              W = d * sc * q - dmin * m  (q4_K)
//
// Warp-level f16 MMAs with the weights from global memory straight into the
// A fragments: every weight byte is read once, by one lane, 16 bytes a load.
// The integer sc * q (or sc * (q - 32)) is formed in binary16: the code bits
// are a subnormal q * 2^-24, one product with 32 * sc makes q * sc * 2^-19.
// For q4_K that is exact (at most 945); for q6_K products beyond 2048 round
// to 11 bits, 2^-12 of themselves and so below the rounding of a 16-bit Y.
// d and dmin multiply in f32 once per super-block. The q4_K min term is one
// MMA per super-block, m_c times the sums of x over the chunks as binary16
// hi/lo pairs.
//
// x is staged once per CTA as binary16 in B-fragment order, each token's 256
// elements scaled by a power of two (largest value in [2^9, 2^10)), so that
// bf16's range is kept and bf16 and f16 inputs are exact down to 2^-26 and 2^-23 of
// the largest. Infinities and NaN stay what they are.
//
// A CTA is 8 warps on R blocks of 16 rows times 8/R parts of K; the parts are
// added through shared memory in a fixed order.
//
// Bound: the latencies of a CTA's walk (its loads, then the sums of its parts) with
// few tiles, instruction issue with many (about 260 instructions per 16 x 256
// weights at 8 tokens; issue 46 % and DRAM 29 % busy at 8 experts of 4096 x 4096),
// before the weight bytes (0.5625 / 0.82 a weight). One token, 8 of 64 q4_K experts
// of 1536 x 2048 with swiglu, 14.2 MB: 8.6 us out of a graph. Persistent CTAs on
// runs of rows, and three CTAs an SM, spilled and were not faster.
#include "moe_internal.cuh"

namespace q6 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = 8;
constexpr int kSmem = 104 * 1024;  // two CTAs an SM

constexpr int kAhead = 4;  // see prefetch_rows()

// Shared bytes of one super-block of 8 * NT staged tokens: x, the chunk-sum
// pairs, the scales.
template <int NT>
constexpr int kSbBytes = 8 * NT * (512 + 32 + 4);
// Super-blocks staged at a time (the partial sums reuse the space).
template <int NT>
constexpr int kSbStage = kSmem / kSbBytes<NT>;

struct Args {
  const uint8_t* plane;
  const void* X;
  long long ldx;
  int gather;
  const int32_t* offsets;
  const int32_t* rows;
  void* Y;
  long long ldy;
  int E, plane_rows, bands, sbs, out, row_groups;
};

__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
constexpr uint32_t kH2_1_16 = 0x2C002C00u;      // (1/16, 1/16)
constexpr uint32_t kH2_32 = 0x50005000u;        // (32, 32)
constexpr uint32_t kH2_m32768 = 0xF800F800u;    // (-32768, -32768)
constexpr uint32_t kH2_m36864 = 0xF880F880u;    // (-36864, -36864)
constexpr uint32_t kH2_m2p19 = 0x80208020u;     // (-2^-19, -2^-19)

// One lane's share of one super-block of 16 rows: rows g and g + 8.
template <int kFmt>
struct Block;
template <>
struct Block<Q6_FMT_Q4K> {
  uint4 q[2][2], head[2];
  __device__ __forceinline__ void load(const uint8_t* tile, int row, int t) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint8_t* p = tile + (row + 8 * r) * 16;
      head[r] = ldg_stream(p);
#pragma unroll
      for (int h = 0; h < 2; ++h) q[r][h] = ldg_stream(p + (1 + 2 * t + h) * 2048);
    }
  }
};
template <>
struct Block<Q6_FMT_Q6K> {
  uint4 q[2][2], high[2];
  uint2 sc[2];
  uint16_t d[2];
  __device__ __forceinline__ void load(const uint8_t* tile, int row, int t) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint8_t* p = tile + (row + 8 * r) * 16;
#pragma unroll
      for (int h = 0; h < 2; ++h) q[r][h] = ldg_stream(p + (2 * t + h) * 2048);
      high[r] = ldg_stream(p + (8 + t) * 2048);
      sc[r] = __ldg(reinterpret_cast<const uint2*>(p + 12 * 2048 + (t >> 1) * 8));
      d[r] = __ldg(reinterpret_cast<const uint16_t*>(tile + 13 * 2048) + row + 8 * r);
    }
  }
};

// Asks for the lines of 16 rows (the first of them row) of a q6_K tile, a line a
// lane: its loads are more and smaller than q4_K's. (Five super-blocks ahead, 16
// experts of 4096 x 11008 in use: q6_K 85.1 us, without 98.8; q4_K 71.2 and 69.4.)
__device__ __forceinline__ void prefetch_rows(const uint8_t* tile, int row, int lane) {
  constexpr int kUnits = 13;  // of 16 bytes a row; then d
  const uint8_t* p = lane < 2 * kUnits ? tile + lane / 2 * 2048 + row * 16 + lane % 2 * 128
                                       : tile + kUnits * 2048 + row * 2;
  if (lane <= 2 * kUnits) asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// acc += one super-block. xs: this super-block's staged x, [chunk][token][run]
// 16-byte units; sums: [token][16] halves (8 hi, 8 lo); scale: [token].
template <int NT>
__device__ __forceinline__ void multiply(const Block<Q6_FMT_Q4K>& b, const uint4* xs,
                                         const uint32_t* sums, const float* scale, int lane,
                                         float (&acc)[NT][4]) {
  const int g = lane >> 2, t = lane & 3;
  uint32_t sc[2][2], mp[2];
  float d[2], dm[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const uint32_t w0 = b.head[r].y, w1 = b.head[r].z, w2 = b.head[r].w;
    sc[r][0] = w0 & 0x3F3F3F3Fu;
    sc[r][1] = (w2 & 0x0F0F0F0Fu) | ((w0 >> 2) & 0x30303030u);
    const uint32_t m0 = w1 & 0x3F3F3F3Fu;
    const uint32_t m1 = ((w2 >> 4) & 0x0F0F0F0Fu) | ((w1 >> 2) & 0x30303030u);
    // mins of chunks 2t and 2t + 1 as halves
    const uint32_t mw = (t < 2 ? m0 : m1) >> (16 * (t & 1));
    mp[r] = hsub2u(__byte_perm(mw, 0x64u, 0x4140u), kH2_1024);
    const float2 dd = unpack2<__half>(b.head[r].x);
    d[r] = dd.x * 524288.0f;  // undoes the 2^-19 of the integers
    dm[r] = dd.y;
  }
  float u[NT][4] = {}, v[NT][4] = {};
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t a[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t w = word4(b.q[r][c / 4], c % 4);
      const uint32_t s1 = __byte_perm(sc[r][c / 4], 0x64u, 0x4040u | (c % 4) << 8 | (c % 4));
      const uint32_t s = hfma2u(s1, kH2_32, kH2_m32768);  // 32 * sc
      const uint32_t s16 = hmul2u(s, kH2_1_16), w8 = w >> 8;  // for codes four bits up
      a[r][0] = hmul2u(w & 0x000F000Fu, s);
      a[r][1] = hmul2u(w & 0x00F000F0u, s16);
      a[r][2] = hmul2u(w8 & 0x000F000Fu, s);
      a[r][3] = hmul2u(w8 & 0x00F000F0u, s16);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint4 x = xs[(c * NT + nt) * 32 + lane];
      const uint32_t a0[4] = {a[0][0], a[1][0], a[0][1], a[1][1]};
      const uint32_t a1[4] = {a[0][2], a[1][2], a[0][3], a[1][3]};
      mma_f16(u[nt], a0, x.x, x.y, u[nt]);
      mma_f16(u[nt], a1, x.z, x.w, u[nt]);
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const uint32_t* s = sums + (nt * 8 + g) * 8;
    const uint32_t am[4] = {mp[0], mp[1], mp[0], mp[1]};
    mma_f16(v[nt], am, s[t], s[4 + t], v[nt]);
    const float2 f = *reinterpret_cast<const float2*>(scale + nt * 8 + 2 * t);
    acc[nt][0] += f.x * (d[0] * u[nt][0] - dm[0] * v[nt][0]);
    acc[nt][1] += f.y * (d[0] * u[nt][1] - dm[0] * v[nt][1]);
    acc[nt][2] += f.x * (d[1] * u[nt][2] - dm[1] * v[nt][2]);
    acc[nt][3] += f.y * (d[1] * u[nt][3] - dm[1] * v[nt][3]);
  }
}

template <int NT>
__device__ __forceinline__ void multiply(const Block<Q6_FMT_Q6K>& b, const uint4* xs,
                                         const uint32_t*, const float* scale, int lane,
                                         float (&acc)[NT][4]) {
  const int t = lane & 3;
  float u[NT][4] = {};
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t a[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t w = word4(b.q[r][c / 4], c % 4);
      const uint32_t hw = word4(b.high[r], c / 2);
      const uint32_t sw = c < 4 ? b.sc[r].x : b.sc[r].y;
      const uint32_t s1 = __byte_perm(sw, 0x64u, 0x4040u | (c % 4) << 8 | (c % 4));
      const uint32_t s = hfma2u(s1, kH2_32, kH2_m36864);  // 32 * sc
      const uint32_t o = hmul2u(s, kH2_m2p19);             // -32 * 2^-24 * 32 * sc
      q6_pairs(w, hw, c % 2, a[r]);
#pragma unroll
      for (int m = 0; m < 4; ++m) a[r][m] = hfma2u(a[r][m], s, o);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint4 x = xs[(c * NT + nt) * 32 + lane];
      const uint32_t a0[4] = {a[0][0], a[1][0], a[0][1], a[1][1]};
      const uint32_t a1[4] = {a[0][2], a[1][2], a[0][3], a[1][3]};
      mma_f16(u[nt], a0, x.x, x.y, u[nt]);
      mma_f16(u[nt], a1, x.z, x.w, u[nt]);
    }
  }
  const float d0 = __half2float(__ushort_as_half(b.d[0])) * 524288.0f;
  const float d1 = __half2float(__ushort_as_half(b.d[1])) * 524288.0f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float2 f = *reinterpret_cast<const float2*>(scale + nt * 8 + 2 * t);
    acc[nt][0] += f.x * (d0 * u[nt][0]);
    acc[nt][1] += f.y * (d0 * u[nt][1]);
    acc[nt][2] += f.x * (d1 * u[nt][2]);
    acc[nt][3] += f.y * (d1 * u[nt][3]);
  }
}

// Stages super-blocks sb0..sb0+count-1 of the `valid` tokens: one warp per
// (token, super-block), 8 elements a lane, kBatch of them in flight. What is
// past `valid` stays unwritten: it only meets columns that are not stored. odd:
// for q4_K set where a token has infinities (see odd_tokens()).
template <typename T, int kFmt, int NT>
__device__ __forceinline__ void stage_x(const Args& a, long long first, int valid, int sb0,
                                        int count, uint4* xs, uint32_t* sums, float* scale,
                                        int* odd) {
  constexpr int kTok = 8 * NT, kBatch = 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* X = static_cast<const T*>(a.X) + lane * 8;
  const int total = valid * count;
  bool mine = false;
  for (int w0 = warp; w0 < total; w0 += kWarps * kBatch) {
    uint4 v[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int w = w0 + b * kWarps;
      if (w >= total) break;
      const int n = w / count, sb = w - n * count;
      const long long r = a.gather ? a.rows[first + n] : first + n;
      v[b] = *reinterpret_cast<const uint4*>(X + r * a.ldx + (sb0 + sb) * 256);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int w = w0 + b * kWarps;
      if (w >= total) break;
      const int n = w / count, sb = w - n * count;
      float f[8];
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = unpack2<T>(word4(v[b], i));
        f[2 * i] = p.x, f[2 * i + 1] = p.y;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(f[i]));
      // non-negative floats order as their bits
      most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
      if (kFmt == Q6_FMT_Q4K && most == __int_as_float(0x7f800000)) mine = true;
      // 2^e with most * 2^-e in [2^9, 2^10), e within [-116, 118] so that both
      // 2^e and 2^-e are normal
      const int e = min(max((int)(__float_as_uint(most) >> 23) - 127 - 9, -116), 118);
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      uint32_t h[4];
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[i] = pack2<__half>(f[2 * i] * down, f[2 * i + 1] * down);
        const float2 p = unpack2<__half>(h[i]);
        s += p.x + p.y;
      }
      xs[((sb * 8 + (lane >> 2)) * kTok + n) * 4 + (lane & 3)] =
          make_uint4(h[0], h[1], h[2], h[3]);
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if ((lane & 3) == 0) {
        __half* p = reinterpret_cast<__half*>(sums + (sb * kTok + n) * 8);
        const __half hi = __float2half_rn(s);
        p[lane >> 2] = hi;
        p[8 + (lane >> 2)] = __float2half_rn(s - __half2float(hi));
      }
      if (lane == 0) scale[sb * kTok + n] = __uint_as_float((uint32_t)(127 + e) << 23);
    }
  }
  if (kFmt == Q6_FMT_Q4K && mine) *odd = 1;
}

// The product of one row of q4_K tiles with a row of x that has infinities: what
// they, and infinite or NaN scales, make of it. The finite rest does not count.
template <typename T>
__device__ __forceinline__ float odd_product(const uint8_t* tiles, int row, int sbs, const T* x) {
  const float inf = __int_as_float(0x7f800000);
  float sum = 0.0f;
  for (int u = 0; u < 32 * sbs; ++u) {  // 8 values each
    const uint8_t* p = tiles + (size_t)(u / 32) * kQ4Tile + row * 16;
    const float2 d = unpack2<__half>(*reinterpret_cast<const uint32_t*>(p));
    const uint4 v = *reinterpret_cast<const uint4*>(x + 8 * u);
    const bool all = !(fabsf(d.x) < inf && fabsf(d.y) < inf);
    const int c = u / 4 % 8, t = u % 4, j = c % 4;
    for (int i = 0; i < 8; ++i) {
      const float2 pair = unpack2<T>(word4(v, i / 2));
      const float f = i % 2 ? pair.y : pair.x;
      if (!all && fabsf(f) < inf) continue;
      const uint32_t w =
          *reinterpret_cast<const uint32_t*>(p + (1 + 2 * t + c / 4) * 2048 + j * 4);
      const uint32_t s = p[4 + j], m = p[8 + j], l = p[12 + j];
      const uint32_t sc = c < 4 ? s & 63 : (l & 15) | (s >> 6) << 4;
      const uint32_t mn = c < 4 ? m & 63 : l >> 4 | (m >> 6) << 4;
      const uint32_t q = (w >> (4 * (i % 2 * 4 + i / 2))) & 15;
      // both terms are exact, so their difference is 0 only where the weight is
      sum += (d.x * (float)(sc * q) - d.y * (float)mn) * f;
    }
  }
  return sum;
}
// The results of q4_K tokens with infinities once more, weight by weight: the MMAs
// sum a code's terms and the min's apart, and where both come out infinite, or a
// code is 0, they make NaN of a weight's infinite product. (A NaN makes NaN of all
// its token's results there as here.) Of items first..last-1 of an expert, this
// CTA's rows.
template <typename T, bool kGlu>
__device__ __forceinline__ void odd_tokens(const Args& a, int expert, long long first,
                                           long long last) {
  const int cols = (kGlu ? 8 : 16) * a.row_groups;
  for (; first < last; ++first) {
    const T* x = static_cast<const T*>(a.X) + (a.gather ? a.rows[first] : first) * a.ldx;
    bool here = false;
    for (int k = threadIdx.x; k < 256 * a.sbs; k += kThreads) here |= isinf(to_f32(x[k]));
    if (!__syncthreads_or(here)) continue;
    for (int c = threadIdx.x; c < cols; c += kThreads) {
      const int m = (int)blockIdx.x * cols + c;
      if (m >= a.out) continue;
      const int row = (int)blockIdx.x * a.row_groups * 16 + (kGlu ? c / 8 * 16 + c % 8 : c);
      const uint8_t* tiles =
          a.plane + ((size_t)expert * a.bands + row / kBand) * (size_t)a.sbs * kQ4Tile;
      float y = odd_product(tiles, row % kBand, a.sbs, x);
      if (kGlu) y = y / (1.0f + __expf(-y)) * odd_product(tiles, row % kBand + 8, a.sbs, x);
      static_cast<T*>(a.Y)[first * a.ldy + m] = from_f32<T>(y);
    }
  }
}

// The products of up to 8 * NT tokens of one expert with this CTA's rows.
template <typename T, int kFmt, bool kGlu, int NT>
__device__ __forceinline__ void run(const Args& a, int expert, long long first, int valid,
                                    uint4* smem, int* odd) {
  constexpr int kTile = kFmt == Q6_FMT_Q4K ? kQ4Tile : kQ6Tile;
  constexpr int kTok = 8 * NT;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int R = a.row_groups, parts = kWarps / R;
  const int rg = warp % R, part = warp / R;
  const int row0 = ((int)blockIdx.x * R + rg) * 16;  // plane row
  const uint8_t* tiles =
      a.plane + ((size_t)expert * a.bands + row0 / kBand) * (size_t)a.sbs * kTile;
  const int in_band = row0 % kBand + (lane >> 2);
  const bool active = row0 < a.plane_rows;
  constexpr int kStage = kSbStage<NT>;
  float acc[NT][4] = {};
  for (int sb0 = 0; sb0 < a.sbs; sb0 += kStage) {
    const int count = min(kStage, a.sbs - sb0);
    uint4* xs = smem;
    uint32_t* sums = reinterpret_cast<uint32_t*>(xs + count * kTok * 32);
    float* scale = reinterpret_cast<float*>(sums + count * kTok * 8);
    Block<kFmt> cur;
    if (active && part < count)
      cur.load(tiles + (size_t)(sb0 + part) * kTile, in_band, lane & 3);
    if (kFmt == Q6_FMT_Q6K && active)
      for (int k = 1; k <= kAhead && part + k * parts < count; ++k)
        prefetch_rows(tiles + (size_t)(sb0 + part + k * parts) * kTile, row0 % kBand, lane);
    if (sb0) __syncthreads();  // the last stage has been read
    stage_x<T, kFmt, NT>(a, first, valid, sb0, count, xs, sums, scale, odd);
    __syncthreads();
    if (active) {
      for (int sb = part; sb < count; sb += parts) {
        Block<kFmt> next;
        if (sb + parts < count)
          next.load(tiles + (size_t)(sb0 + sb + parts) * kTile, in_band, lane & 3);
        if (kFmt == Q6_FMT_Q6K && sb + (kAhead + 1) * parts < count)
          prefetch_rows(tiles + (size_t)(sb0 + sb + (kAhead + 1) * parts) * kTile, row0 % kBand,
                        lane);
        multiply<NT>(cur, xs + sb * kTok * 32, sums + sb * kTok * 8, scale + sb * kTok, lane, acc);
        cur = next;
      }
    }
  }
  __syncthreads();
  // partial sums [part][token][R * 16 + 4]
  float* red = reinterpret_cast<float*>(smem);
  const int ld = R * 16 + 4;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float* p = red + ((size_t)part * kTok + nt * 8 + 2 * (lane & 3)) * ld + rg * 16 + (lane >> 2);
    p[0] = acc[nt][0];
    p[ld] = acc[nt][1];
    p[8] = acc[nt][2];
    p[ld + 8] = acc[nt][3];
  }
  __syncthreads();
  T* Y = static_cast<T*>(a.Y);
  const int cols = kGlu ? R * 8 : R * 16;
  for (int i = threadIdx.x; i < valid * cols; i += kThreads) {
    const int n = i / cols, c = i % cols;
    const int m = (int)blockIdx.x * cols + c;
    const float* p = red + n * ld + (kGlu ? c / 8 * 16 + c % 8 : c);
    float y = 0.0f, up = 0.0f;
    for (int k = 0; k < parts; ++k) {
      y += p[(size_t)k * kTok * ld];
      if (kGlu) up += p[(size_t)k * kTok * ld + 8];
    }
    if (kGlu) y = y / (1.0f + __expf(-y)) * up;
    if (m < a.out) Y[(first + n) * a.ldy + m] = from_f32<T>(y);
  }
  __syncthreads();
}

template <typename T, int kFmt, bool kGlu>
__device__ __forceinline__ void experts_few(const Args& a) {
  extern __shared__ uint4 smem[];
  __shared__ int odd;
  if (kFmt == Q6_FMT_Q4K) {
    if (threadIdx.x == 0) odd = 0;
    __syncthreads();
  }
  griddep_wait();
  griddep_launch_dependents();
  // the blockIdx.y-th expert that has items
  const int lane = threadIdx.x & 31;
  int left = blockIdx.y, expert = -1;
  for (int e0 = 0; e0 < a.E; e0 += 32) {
    const int e = e0 + lane;
    const unsigned m =
        __ballot_sync(0xffffffffu, e < a.E && a.offsets[e + 1] > a.offsets[e]);
    const int c = __popc(m);
    if (left < c) {
      expert = e0 + __fns(m, 0, left + 1);
      break;
    }
    left -= c;
  }
  if (blockIdx.y == 0) {  // items of no expert: zeros
    const int cols = (kGlu ? 8 : 16) * a.row_groups, m0 = (int)blockIdx.x * cols;
    const long long i0 = a.offsets[a.E], i1 = a.offsets[a.E + 1];
    for (long long i = i0 * cols + threadIdx.x; i < i1 * cols; i += kThreads)
      if (m0 + (int)(i % cols) < a.out)
        static_cast<T*>(a.Y)[i / cols * a.ldy + m0 + i % cols] = from_f32<T>(0.0f);
  }
  if (expert < 0) return;
  const long long i0 = a.offsets[expert];
  int left_items = (int)(a.offsets[expert + 1] - i0);
  for (long long first = i0; left_items > 0;) {
    if (left_items <= 8) {
      run<T, kFmt, kGlu, 1>(a, expert, first, left_items, smem, &odd);
      break;
    }
    const int n = min(left_items, 16);
    run<T, kFmt, kGlu, 2>(a, expert, first, n, smem, &odd);
    first += n;
    left_items -= n;
  }
  if (kFmt == Q6_FMT_Q4K && odd) odd_tokens<T, kGlu>(a, expert, i0, a.offsets[expert + 1]);
}

// Two kernels, for the arguments: as a grid constant they cost q6_K 15.9 instead of
// 13.7 us (16 items over 32 experts of 2056 x 1536), as plain ones q4_K, which has
// odd_tokens() behind it, 25.1 instead of 22.0 us (8 over 8 of 4096 x 4096).
template <typename T, bool kGlu>
__global__ void __launch_bounds__(kThreads, 2)
experts_few_q4_kernel(const __grid_constant__ Args a) {
  experts_few<T, Q6_FMT_Q4K, kGlu>(a);
}
template <typename T, bool kGlu>
__global__ void __launch_bounds__(kThreads, 2) experts_few_q6_kernel(const Args a) {
  experts_few<T, Q6_FMT_Q6K, kGlu>(a);
}

typedef void (*Kernel)(const Args);
template <typename T>
Kernel pick_t(int fmt, int swiglu) {
  if (fmt == Q6_FMT_Q4K)
    return swiglu ? experts_few_q4_kernel<T, true> : experts_few_q4_kernel<T, false>;
  return swiglu ? experts_few_q6_kernel<T, true> : experts_few_q6_kernel<T, false>;
}
Kernel pick(int type, int fmt, int swiglu) {
  return type == Q6_TYPE_BF16 ? pick_t<__nv_bfloat16>(fmt, swiglu) : pick_t<__half>(fmt, swiglu);
}

}  // namespace

cudaError_t experts_few_prepare() {
  for (int type : {Q6_TYPE_BF16, Q6_TYPE_F16})
    for (int fmt : {Q6_FMT_Q4K, Q6_FMT_Q6K})
      for (int glu : {0, 1}) {
        const cudaError_t e = cudaFuncSetAttribute(
            pick(type, fmt, glu), cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
      }
  return cudaSuccess;
}

cudaError_t launch_experts_few(const ExpertCall& c, cudaStream_t s) {
  Args a;
  a.plane = c.plane;
  a.X = c.X, a.ldx = c.ldx, a.gather = c.gather;
  a.offsets = c.offsets, a.rows = c.rows;
  a.Y = c.Y, a.ldy = c.ldy;
  a.E = c.E, a.plane_rows = c.g.rows, a.bands = c.g.bands, a.sbs = c.g.sbs, a.out = c.g.out;
  const unsigned experts = (unsigned)(c.items < c.E ? c.items : c.E);
  // the fewest rows a CTA with which all CTAs run at a time (two an SM)
  int R = 1;
  while (R < 8 && (size_t)experts * (size_t)((c.g.rows + 16 * R - 1) / (16 * R)) > 2 * 152) R *= 2;
  a.row_groups = R;
  const dim3 grid((unsigned)((c.g.rows + 16 * R - 1) / (16 * R)), experts);
  // what the launch needs of the shared memory: one stage of x, or the sums
  const int nt = c.items > 8 ? 2 : 1;
  const int sb_bytes = nt == 2 ? kSbBytes<2> : kSbBytes<1>;
  int smem = sb_bytes * c.g.sbs;
  if (smem > kSmem) smem = kSmem;
  const int sums = kWarps / R * 8 * nt * (R * 16 + 4) * 4;
  if (smem < sums) smem = sums;
  return launch_pdl(pick(c.type, c.fmt, c.swiglu), grid, dim3(kThreads), (size_t)smem, s, a);
}

}  // namespace q6
