// Grouped K-quant expert products on the 5th-generation tensor cores, for
// experts with many tokens.
//
//   Y[i][m] = sum_k W[e(i)][m][k] x[t(i)][k]
//
// A pair of CTAs (cluster of two, cta_group::2) computes a tile of 256 plane
// rows of one expert (MMA M; 128 rows, one TMEM lane each, a CTA) by up to 256
// of its items (MMA N; each CTA loads half of their x). Sharing x halves what
// shared memory has to take in and hand out: one CTA alone on 128 x 256 moves
// 64 KB in and out of it for 512 cycles of MMA, which is all it can
// (measured, 8192 items of 11008 x 4096: 621 us alone).
//
// The weights are dequantised inside the kernel, once per tile: thread =
// weight row, binary16 pairs, the result stored straight into TMEM, where the
// MMA takes its A operand from. Packed weights are all that memory and shared
// memory ever see. A code is the binary16 subnormal q * 2^-24 and a weight one
// fused multiply-add of it with sc * d and -dmin * m, all times a power of two of
// the row (the largest possible weight of a row just below 2^-5): what is rounded
// to 11 bits is sc * d, dmin * m and the weight, each an eighth of the rounding of
// a bf16 Y. That leaves binary16 2^9 of range above its smallest normal number, so
// 32 rows of which one has super-blocks whose weights are less than 2^-7 of its
// largest (marked when packed) go another way: sc * q exact, times d in the fused
// multiply-add, 2^15 times larger. (Rates, cycles a warp instruction of one
// scheduler: binary16 pairs 2, integer logic and shifts 2, on two pipes; f32 1. That
// way is 3.7 instead of 2.8 instructions a pair, and 8 experts of 4096 x 4096 took
// 28.8 instead of 27.0 us.) The smallest step there is 2^-33 of a row's largest
// possible weight: half of it is 2^-12 of a super-block's down to 2^-22 of the row's.
// For a binary16 Y that would show, so there the weight is rounded once (q4_K in f32,
// 2.6 instructions a weight; q6_K with sc * d in two terms, 3.4).
// In a binary16 silu(gate) * up the roundings of both products would still
// add up to 1.7 times that of Y; there a weight is a pair of binary16 values
// in two A slots, and every x tile meets both.
//
// x comes as binary16 in item order: bf16 rows scaled by a power of two (exact
// down to 2^-31 of the row's largest value), gathered ones copied, by a kernel
// before this one; binary16 rows that are in order are read where they are.
// TMA loads them as 128-byte-swizzled K-major tiles. (Gathering with TMA's own
// row gather, 4 rows a request, was measured at about 60 cycles a request,
// 4000 for the 256 rows of a stage whose MMAs take 512.)
//
// Warp roles (20 warps, persistent CTAs, one per SM):
//   0      loads x
//   1      in CTA 0, issues the pair's MMAs
//   2      TMEM allocation
//   3      streams the packed weights, one super-block a stage
//   4-11   dequantise: warps 4-7 the even, 8-11 the odd super-blocks. A group
//          waits, loads and hands over for about as long as it calculates, and
//          the other's calculation fills that time; when both worked on the
//          halves of one super-block they did everything at the same time (1350
//          instead of 1050 cycles a super-block with few items). Sixteen warps
//          instead of eight, by halves or quarters, with 72 registers: not faster.
//   12-19  epilogue: warps 12-15 items 0-127 of a tile, 16-19 the others (or
//          every other tile of up to 128 items)
// TMEM: columns 0-255 two accumulators of 128 items (or one of 256), 256-511
// four A slots of 128 of K.
// The walk is in units: 128 of K for tiles of more than 128 items (or weights
// in pairs), 256 for others. A unit has one x stage and one or two A slots; one
// barrier says that all of it is there (both CTAs' copies and dequantised halves), another that
// its MMAs are through. (A wait costs the MMA warp about 120 cycles and a
// commit 150 or more, a unit's MMAs at 128 items 1024: with separate barriers
// for x and A and 128 of K each, 1023 tokens over 64 experts took 119 us.)
// Bound: the MMAs at 256 items a tile (8192 bf16 items of q4_K experts of 11008 x
// 4096, 739 GFLOP: 500 us, 1.48 PFLOP/s; its tensor pipe 76 % busy at 100 us), the
// dequantising warps at few (132 items over 32 q6_K experts of 2056 x 1536, 83 MB:
// 29.5 us), where issue is 51 % and DRAM 41 % busy: about 1050 cycles a super-block
// against 512 of MMA at 64 items.
// Every wait is bounded (see q6_internal.cuh), and the pair meets once more
// before either CTA leaves.
#include "moe_internal.cuh"
#include "tc_pair.cuh"

namespace q6 {
namespace {

constexpr int kThreads = 640;
constexpr int kTileN = 256;
// Units in flight, and those with their x in shared memory; packed super-blocks
// there, of either format what is left. (With a fourth x stage q6_K keeps two
// super-blocks, half of what HBM's latency wants: 8 experts of 4096 x 4096 with
// 32 items each took 43.5 instead of 34.7 us.)
constexpr int kUnits = 4, kXStages = 3, kXStage = 32 * 1024;
template <int kFmt>
constexpr int kWStages = kFmt == Q6_FMT_Q4K ? 5 : 4;
constexpr int kMaxWStages = 5;
constexpr int kASlots = 4, kACols = 64, kACol0 = 256;
constexpr int kTmemCols = 512;

enum : uint32_t { kSiteReady = 32, kSiteDone, kSiteWEmpty, kSiteWFull, kSiteDEmpty, kSiteDFull,
                  kSiteDrain };

struct Bars {
  uint64_t ready[kUnits], done[kUnits];
  uint64_t w_full[kMaxWStages], w_empty[kMaxWStages];
  uint64_t d_full[2], d_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
// Arrivals that make a unit ready: the x copies' opening, and the pair's eight
// warps that dequantise it.
constexpr int kReadyArrivals = 9;

struct Args {
  const uint8_t* plane;
  const float* scale;  // 2^e per plane row
  const float* xscale;  // per item, or NULL: 1
  const int32_t* offsets;
  void* Y;
  long long ldy;
  int E, bands, sbs, out;
  int vec;  // Y and its rows are 16-byte aligned
  int early;  // the kernel before is expert_rows_kernel: only x depends on it
};

template <int kFmt>
constexpr int kWTile = kFmt == Q6_FMT_Q4K ? kQ4Tile : kQ6Tile;
constexpr int kMaxSorted = 256;  // experts whose tiles are put in order of size
constexpr int kOutWarp = 2048;  // epilogue staging of a warp: 32 items of 64 bytes
template <int kFmt>
constexpr int kSmemBytes = 1024 + kXStages * kXStage + kWStages<kFmt> * kWTile<kFmt> + 8 * kOutWarp +
                           2 * (kMaxGroups + 1) * 4 + kMaxSorted + (int)sizeof(Bars);

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]^T over the CTA pair, kind::f16.
__device__ __forceinline__ void umma_f16_pair(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 bd;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 bd, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], bd, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kSw128DescHi)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 16 TMEM lanes x 32 columns as four MMA accumulator fragments: r[4 j + e] is
// row lane / 4 (+ 8 for e >= 2), column 8 j + 2 (lane % 4) + e % 2.
__device__ __forceinline__ void tmem_ld_frag(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tmem_wait_frag(uint32_t (&a)[16], uint32_t (&b)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]), "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]), "+r"(a[12]), "+r"(a[13]), "+r"(a[14]), "+r"(a[15]),
                 "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]), "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7]), "+r"(b[8]), "+r"(b[9]), "+r"(b[10]), "+r"(b[11]), "+r"(b[12]), "+r"(b[13]), "+r"(b[14]), "+r"(b[15])
               :
               : "memory");
}
// Four transposed 8 x 8 tiles of 16-bit values: lane l gives the address of
// row l % 8 of tile l / 8.
__device__ __forceinline__ void store_tiles_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                              uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// ------------------------------------------------------------ dequantising ---
constexpr uint32_t kH2_2m11 = 0x10001000u, kH2_2m15 = 0x02000200u, kH2_512 = 0x60006000u,
                   kH2_256 = 0x5C005C00u, kH2_m2p19 = 0x80208020u, kH2_1_16 = 0x2C002C00u,
                   kH2_4 = 0x44004400u, kH2_4_8th = 0x44204420u;  // 4 + 32 / 256

// A byte of a word as a binary16 pair, plus 1024.
__device__ __forceinline__ uint32_t byte_h2(uint32_t w, int i) {
  return __byte_perm(w, 0x64u, 0x4040u | i << 8 | i);
}
// v as a binary16 pair (both halves).
__device__ __forceinline__ uint32_t splat_h2(float v) {
  const __half2 h = __float2half2_rn(v);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A code as f32: in bits p.. of x, with the exponent of 2^(23 - p) above it, it is
// the float 2^(23 - p) + code.
__device__ __forceinline__ float code_f32(uint32_t x, uint32_t mask, uint32_t magic) {
  return __uint_as_float((x & mask) | magic);
}
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma_f2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t round_f2(uint64_t v) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
  return pack2<__half>(x, y);
}
__device__ __forceinline__ float byte_f32(uint32_t w, int i) {
  return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u | i)) - 8388608.0f;
}

// One row's half (128 of K) of a super-block.
template <int kFmt>
struct Half;
template <>
struct Half<Q6_FMT_Q4K> {
  uint4 q[4];
  uint32_t sc, mn, d, dm;
  float df, dmf;
  __device__ __forceinline__ void load(const uint8_t* tile, int row, int h, float inv, bool wide) {
    const uint4* p = reinterpret_cast<const uint4*>(tile) + row;
    const uint4 head = p[0];
#pragma unroll
    for (int t = 0; t < 4; ++t) q[t] = p[(1 + 2 * t + h) * kBand];
    const float2 dd = unpack2<__half>(head.x);
    df = dd.x * inv, dmf = -dd.y * inv;
    d = splat_h2(df * (wide ? 32768.0f : 512.0f)), dm = splat_h2(dmf * (wide ? 2048.0f : 1.0f));
    sc = h ? (head.w & 0x0F0F0F0Fu) | ((head.y >> 2) & 0x30303030u) : head.y & 0x3F3F3F3Fu;
    mn = h ? ((head.w >> 4) & 0x0F0F0F0Fu) | ((head.z >> 2) & 0x30303030u) : head.z & 0x3F3F3F3Fu;
  }
  // Chunk cc of the half (32 of K) as 16 words.
  template <bool kWide>
  __device__ __forceinline__ void expand(int cc, uint32_t (&out)[16]) const {
    // sc * d * 2^9, or sc * 2^9
    const uint32_t s = hmul2u(hsub2u(byte_h2(sc, cc), kH2_1024), kWide ? kH2_512 : d);
    const uint32_t s16 = hmul2u(s, kH2_1_16);  // for codes four bits up
    // -dmin * m (dm, which kWide makes 2^11 larger, is no subnormal either way)
    uint32_t m = hsub2u(byte_h2(mn, cc), kH2_1024);
    m = kWide ? hmul2u(hmul2u(m, kH2_2m11), dm) : hmul2u(hmul2u(m, dm), kH2_2m15);
    auto weight = [&](uint32_t code, uint32_t by) {
      return kWide ? hfma2u(hmul2u(code, by), d, m) : hfma2u(code, by, m);
    };
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t w = word4(q[t], cc), w8 = w >> 8;
      out[4 * t] = weight(w & 0x000F000Fu, s);
      out[4 * t + 1] = weight(w & 0x00F000F0u, s16);
      out[4 * t + 2] = weight(w8 & 0x000F000Fu, s);
      out[4 * t + 3] = weight(w8 & 0x00F000F0u, s16);
    }
  }
  // In f32, rounded once. The offsets of the codes go with the min (rounded to
  // at most 2^-12 of the scale).
  __device__ __forceinline__ void expand_once(int cc, uint32_t (&out)[16]) const {
    expand_f32<false>(cc, out, out);
  }
  // In f32, as two binary16 values (the min beside a code without an offset).
  __device__ __forceinline__ void expand_pair(int cc, uint32_t (&out)[16],
                                              uint32_t (&rest)[16]) const {
    expand_f32<true>(cc, out, rest);
  }
  template <bool kTwo>
  __device__ __forceinline__ void expand_f32(int cc, uint32_t (&out)[16],
                                             uint32_t (&rest)[16]) const {
    const float s = df * byte_f32(sc, cc), m = dmf * byte_f32(mn, cc);
    const float c11 = fmaf(-4096.0f, s, m), c15 = fmaf(-256.0f, s, m), c19 = fmaf(-16.0f, s, m),
                c12 = fmaf(-2048.0f, s, m);
    const uint64_t ss = f2(s, s);
    auto weight = [&](float lo, float hi, float offset, float c, int i) {
      if (kTwo) {  // the code alone is exact, and so are few bits times s: one rounding, at 2^-24
        const uint64_t v = fma_f2(f2(lo - offset, hi - offset), ss, f2(m, m));
        float a, b;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
        out[i] = pack2<__half>(a, b);
        const float2 h = unpack2<__half>(out[i]);
        rest[i] = pack2<__half>(a - h.x, b - h.y);
      } else {
        out[i] = round_f2(fma_f2(f2(lo, hi), ss, f2(c, c)));
      }
    };
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t w = word4(q[t], cc), a = w << 11, b = w >> 5, e = w >> 16;
      weight(code_f32(a, 0x7800u, 0x45800000u), code_f32(b, 0x7800u, 0x45800000u), 4096.0f, c11, 4 * t);
      weight(code_f32(a, 0x78000u, 0x43800000u), code_f32(b, 0x78000u, 0x43800000u), 256.0f, c15, 4 * t + 1);
      weight(code_f32(a, 0x780000u, 0x41800000u), code_f32(b, 0x780000u, 0x41800000u), 16.0f, c19, 4 * t + 2);
      weight(code_f32(w, 0xF000u, 0x45000000u), code_f32(e, 0xF000u, 0x45000000u), 2048.0f, c12, 4 * t + 3);
    }
  }
};
template <>
struct Half<Q6_FMT_Q6K> {
  uint4 q[4];
  uint2 high[4];
  uint32_t sc[2], d;
  float df;
  __device__ __forceinline__ void load(const uint8_t* tile, int row, int h, float inv, bool wide) {
    const uint4* p = reinterpret_cast<const uint4*>(tile) + row;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      q[t] = p[(2 * t + h) * kBand];
      high[t] = reinterpret_cast<const uint2*>(p + (8 + t) * kBand)[h];
    }
    const uint32_t* s = reinterpret_cast<const uint32_t*>(p + 12 * kBand);
    sc[0] = s[h], sc[1] = s[2 + h];
    df = __half2float(reinterpret_cast<const __half*>(tile + 13 * 2048)[row]) * inv;
    d = splat_h2(df * (wide ? 65536.0f : 512.0f));
  }
  template <bool kWide>
  __device__ __forceinline__ void expand(int cc, uint32_t (&out)[16]) const {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {  // runs 0, 1 and 2, 3 of the chunk
      // sc * d * 2^9, or sc * 2^8
      const uint32_t s = hmul2u(hsub2u(byte_h2(sc[sub], cc), kH2_1152), kWide ? kH2_256 : d);
      const uint32_t o = hmul2u(s, kH2_m2p19);  // -32 * 2^-24 * s
#pragma unroll
      for (int t = 2 * sub; t < 2 * sub + 2; ++t) {
        uint32_t v[4];
        q6_pairs(word4(q[t], cc), cc < 2 ? high[t].x : high[t].y, cc % 2, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = hfma2u(v[i], s, o);
          out[4 * t + i] = kWide ? hmul2u(w, d) : w;
        }
      }
    }
  }
  // The scale sc * d as two binary16 terms: their sum and so the weight is
  // rounded once. (256 times larger, and the code as much smaller, so that the
  // second term of a small super-block keeps its bits.)
  __device__ __forceinline__ void expand_once(int cc, uint32_t (&out)[16]) const {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const float s = 256.0f * df * (byte_f32(sc[sub], cc) - 128.0f);
      const uint32_t hi = splat_h2(s), lo = splat_h2(s - unpack2<__half>(hi).x);
#pragma unroll
      for (int t = 2 * sub; t < 2 * sub + 2; ++t) {
        uint32_t v[4];
        q6_pairs(word4(q[t], cc), cc < 2 ? high[t].x : high[t].y, cc % 2, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t c = hsub2u(v[i] | kH2_4, kH2_4_8th);  // (q - 32) / 256
          out[4 * t + i] = hfma2u(c, hi, hmul2u(c, lo));
        }
      }
    }
  }
  // The weight and what it was rounded by.
  __device__ __forceinline__ void expand_pair(int cc, uint32_t (&out)[16],
                                              uint32_t (&rest)[16]) const {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const float s = 256.0f * df * (byte_f32(sc[sub], cc) - 128.0f);
      const uint32_t hi = splat_h2(s), lo = splat_h2(s - unpack2<__half>(hi).x);
#pragma unroll
      for (int t = 2 * sub; t < 2 * sub + 2; ++t) {
        uint32_t v[4];
        q6_pairs(word4(q[t], cc), cc < 2 ? high[t].x : high[t].y, cc % 2, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t c = hsub2u(v[i] | kH2_4, kH2_4_8th);  // (q - 32) / 256
          const uint32_t w = hfma2u(c, hi, hmul2u(c, lo));
          out[4 * t + i] = w;
          // c * hi - w is exact (17 bits less the upper 11)
          rest[4 * t + i] = hfma2u(c, lo, hfma2u(c, hi, w ^ 0x80008000u));
        }
      }
    }
  }
};

// x / (1 + exp(-x)), within the exponential's 2 + 1.2 |x| and the division's 2 units of
// 2^-23: 2^-20 where x is above -3, 2^-16 at -87 (0 below that, where it is under 2^-118).
__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.0f + __expf(-x)); }

// ---------------------------------------------------------------- schedule ---
struct Tile {
  int expert, pair, n;  // pair of bands; n: MMA N, a multiple of 32
  long long first;      // first item
  int count;            // items
};
__device__ __forceinline__ int tiles_of(int count) { return (count + kTileN - 1) / kTileN; }

// Items of an expert's tiles: equal parts, in steps of 32 (their last may hold
// less, but never nothing).
__device__ __forceinline__ int tile_items(int count) {
  const int parts = tiles_of(count);
  return parts ? ((count + parts - 1) / parts + 31) / 32 * 32 : 0;
}
// Tile t of the list ordered by (expert, item tile, band pair); start[i] is the
// number of (expert, item tile)s before the i-th expert, which is i or, if sorted,
// order[i]. Nothing (n = 0) past the last tile.
__device__ __forceinline__ Tile tile_at(const Args& a, const int* start, const int* offs,
                                        const uint8_t* order, bool sorted, int t, int total) {
  Tile r = {};
  if (t >= total) return r;
  const int pairs = (a.bands + 1) / 2;
  const int item_tile = t / pairs;
  int lo = 0, hi = a.E;  // start[lo] <= item_tile < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (start[mid] <= item_tile) lo = mid;
    else hi = mid;
  }
  r.expert = sorted ? order[lo] : lo, r.pair = t % pairs;
  const int begin = offs[r.expert], count = offs[r.expert + 1] - begin, j = item_tile - start[lo];
  r.n = tile_items(count);
  r.first = (long long)begin + (long long)j * r.n;
  r.count = min(r.n, count - j * r.n);
  return r;
}
// This CTA's band of the pair; past an odd number of bands the last one again,
// whose result is not stored.
__device__ __forceinline__ int band_of(const Args& a, int pair, int rank) {
  return min(2 * pair + rank, a.bands - 1);
}
// A CTA's n / 2 rows of x come as one box of 16, 32, 64 or 128 rows (the rows
// past n / 2 are loaded and not used: one request a block is worth more than
// the bytes; requests by several lanes took about 150 cycles each).
__device__ __forceinline__ int box_of(int n) { return n > 128 ? 3 : n > 64 ? 2 : n > 32 ? 1 : 0; }
// Whether a weight is two binary16 values.
template <typename T, bool kGlu>
constexpr bool kPair = __is_same(T, __half) && kGlu;
// log2 of a unit's 64-of-K blocks.
template <bool kTwo>
__device__ __forceinline__ int unit_shift(int n) { return kTwo || n > 128 ? 1 : 2; }

// The MMAs of one tile, by the whole MMA warp; kShift = unit_shift(n). kTwo:
// weights in pairs, the second ones in the next A slot.
struct MmaState {
  int unit, a;  // units and A slots used so far
};
template <int kShift, bool kTwo>
__device__ __forceinline__ bool tile_mmas(MmaState& st, Bars* bars, const uint8_t* xring,
                                          uint32_t tmem, uint32_t d_tmem, int n, int sbs,
                                          volatile int* abort_flag, unsigned int* status) {
  // f16 operands, f32 accumulation, M = 256
  const uint32_t idesc = idesc_f16_f32(256, n);
  const uint32_t x_block = (uint32_t)(16 << box_of(n)) * 128 >> 4;  // in descriptor units
  const uint32_t x0 = sw128_desc_lo(smem_u32(xring));
  const int units = 4 * sbs >> kShift;
  for (int u = 0; u < units; ++u) {
    const int slot = st.unit % kUnits;
    if (!mbar_wait_warp(&bars->ready[slot], (st.unit / kUnits) & 1, abort_flag, status, kSiteReady))
      return false;
    tc_fence_after();
    if (elect_one()) {
      const uint32_t b = x0 + st.unit % kXStages * (kXStage >> 4);
      // two A slots of a unit are neighbours, the first an even one
      const uint32_t at = tmem + (uint32_t)(kACol0 + st.a % kASlots * kACols);
#pragma unroll
      for (int i = 0; i < 4 << kShift; ++i) {
        const uint32_t bi = b + (i / 4) * x_block + 2 * (i % 4);
        umma_f16_pair(d_tmem, at + 8 * i, bi, idesc, (uint32_t)(u > 0 || i > 0));
        if (kTwo) umma_f16_pair(d_tmem, at + kACols + 8 * i, bi, idesc, 1u);
      }
      commit_pair(&bars->done[slot]);
    }
    __syncwarp();
    ++st.unit;
    st.a += kTwo ? 2 : kShift;
  }
  return true;
}

template <typename T, int kFmt, bool kGlu>
__global__ void __launch_bounds__(kThreads, 1)
experts_tc_kernel(const __grid_constant__ RowMaps maps, const Args a, unsigned int* status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* xring = smem;
  uint8_t* wring = smem + kXStages * kXStage;
  uint8_t* out_stage = wring + kWStages<kFmt> * kWTile<kFmt>;
  int* start = reinterpret_cast<int*>(out_stage + 8 * kOutWarp);
  int* offs = start + kMaxGroups + 1;  // a copy of the offsets
  uint8_t* order = reinterpret_cast<uint8_t*>(offs + kMaxGroups + 1);
  Bars* bars = reinterpret_cast<Bars*>(order + kMaxSorted);
  static_assert(2 * (kMaxGroups + 1) * 4 % 8 == 0, "barriers are 8-byte aligned");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), cluster = blockIdx.x / 2, clusters = gridDim.x / 2;
  volatile int* abort_flag = &bars->abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(&bars->ready[i], kReadyArrivals);  // used in CTA 0
      mbar_init(&bars->done[i], 1);
    }
    for (int i = 0; i < kWStages<kFmt>; ++i) {
      mbar_init(&bars->w_full[i], 1);
      mbar_init(&bars->w_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->d_full[i], 1);
      mbar_init(&bars->d_empty[i], 8);
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    mbar_fence_init();
    for (int i = 0; i < RowMaps::kCount; ++i) tma_prefetch_desc(&maps.box[i]);
  }
  if (warp == 2) {
    tmem_alloc_pair(&bars->tmem_base, kTmemCols);
  }
  // The kernel before has passed its own wait once this one runs, so all before it
  // is in memory: where it made nothing but the rows of x, only their readers wait.
  if (!a.early) griddep_wait();
  griddep_launch_dependents();
  // Tiles of more than 128 items (there are such with more than 128 items an expert)
  // take longer the more they have, others all the same, by their weights: with any
  // of them the largest come first. (8184 items unevenly over 64 experts of 2816 x
  // 2048: 112 us, in the experts' order 114 to 120; 2048 over 8 of 4096 x 4096 61 and
  // 67.) Not with more than 256 experts: their ranks, found by comparing each with
  // all, would take microseconds, and shared memory has no room for a longer order.
  bool large = false;
  for (int e = threadIdx.x; e <= a.E; e += kThreads) {
    const int begin = a.offsets[e];
    offs[e] = begin;
    large |= e < a.E && a.offsets[e + 1] - begin > 128;
  }
  const bool sorted = __syncthreads_or(large) && a.E <= kMaxSorted;
  if (sorted) {
    const int e = threadIdx.x, n = e < a.E ? tile_items(offs[e + 1] - offs[e]) : 0;
    if (e < a.E) start[e] = n;
    __syncthreads();
    if (e < a.E) {
      int before = 0;
      for (int i = 0; i < a.E; ++i) before += start[i] > n || (start[i] == n && i < e);
      order[before] = (uint8_t)e;
    }
    __syncthreads();
  }
  if (warp == 3) {  // start[]: the running number of (expert, item tile) pairs
    int run = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int at = sorted && e < a.E ? order[e] : e;
      const int v = e < a.E ? tiles_of(offs[at + 1] - offs[at]) : 0;
      int x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (e < a.E) start[e] = run + x - v;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) start[a.E] = run;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const int total = start[a.E] * ((a.bands + 1) / 2);
  // Each role works out its next tile while it has one: between two tiles that
  // would stand still for 1300 cycles. The pairs take the list in turn, with the
  // largest tiles first every second time in reverse, so that their sums come out
  // alike; the last time is not, for the pairs that started first have the rest (the
  // last of a launch start about a microsecond later).
  int pass = 0;
  const int odd = sorted ? (total + clusters - 1) / clusters % 2 : 0;  // passes in all
  auto number = [&] {
    const bool reverse = sorted && pass % 2 == odd;
    return pass * clusters + (reverse ? clusters - 1 - cluster : cluster);
  };
  Tile next = tile_at(a, start, offs, order, sorted, number(), total);
  auto take = [&] {
    const Tile w = next;
    ++pass;
    next = tile_at(a, start, offs, order, sorted, number(), total);
    return w;
  };
  bool ok = true;

  constexpr bool kTwo = kPair<T, kGlu>;
  if (warp == 0) {
    // --------------------------------------------------------------- load x --
    griddep_wait();
    int g = 0;  // units opened
    while (next.n && ok) {
      const Tile w = take();
      const int rows = w.n / 2;  // this CTA's
      const int box = box_of(w.n);
      const int shift = unit_shift<kTwo>(w.n);
      const int row0 = __shfl_sync(0xffffffffu, (int)w.first + rank * rows, 0);
      const int block = (16 << box) * 128;
      for (int k = 0; k < 4 * a.sbs; k += 1 << shift) {
        const int slot = g % kUnits, last = g - kXStages;  // last: the unit before in this x stage
        if (last >= 0 && !(ok = mbar_wait_warp(&bars->done[last % kUnits], (last / kUnits) & 1,
                                               abort_flag, status, kSiteDone)))
          break;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&bars->ready[slot], (uint32_t)(2 * block) << shift);
          for (int b = 0; b < 1 << shift; ++b)
            tma_load_2d_pair(xring + g % kXStages * kXStage + b * block, &maps.box[box],
                             &bars->ready[slot], (k + b) * 64, row0);
        }
        __syncwarp();
        ++g;
      }
    }
    // the last units' MMAs are through, and this CTA has been told, before it
    // leaves
    for (int k = g > kUnits ? g - kUnits : 0; k < g && ok; ++k)
      ok = mbar_wait_warp(&bars->done[k % kUnits], (k / kUnits) & 1, abort_flag, status, kSiteDone);
    if (!ok && lane == 0) {
      // Copies in flight land before the CTA exits. They count on a barrier
      // that other arrivals complete too, so they are given 1 ms.
      for (const long long t0 = clock64(); clock64() - t0 < 2100000;) {
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------- packed weights --
    int slot = 0, round = 0, g = 0;  // g: stages filled
    while (next.n && ok) {
      const Tile w = take();
      const size_t band = (size_t)w.expert * a.bands + band_of(a, w.pair, rank);
      const uint8_t* src = a.plane + __shfl_sync(0xffffffffu, band, 0) * (size_t)a.sbs * kWTile<kFmt>;
      for (int sb = 0; sb < a.sbs; ++sb) {
        if (!(ok = mbar_wait_warp(&bars->w_empty[slot], (round & 1) ^ 1, abort_flag, status,
                                  kSiteWEmpty)))
          break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&bars->w_full[slot], kWTile<kFmt>);
          bulk_load(wring + slot * kWTile<kFmt>, src, kWTile<kFmt>, &bars->w_full[slot]);
        }
        __syncwarp();
        src += kWTile<kFmt>;
        ++g;
        if (++slot == kWStages<kFmt>) slot = 0, ++round;
      }
    }
    if (!ok && lane == 0) {
      volatile int no_abort = 0;
      for (int k = g > kWStages<kFmt> ? g - kWStages<kFmt> : 0; k < g; ++k)
        mbar_wait_bounded(&bars->w_full[k % kWStages<kFmt>], (k / kWStages<kFmt>) & 1, &no_abort, status,
                          kSiteWFull);
    }
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------------ MMA --
    // (Issued from one lane's own branch, 64 of K took 700 cycles.)
    MmaState st = {0, 0};
    int turn = 0, uses0 = 0, uses1 = 0;
    while (next.n && ok) {
      const int n = (int)__reduce_max_sync(0xffffffffu, (unsigned)take().n);
      const bool both = n > 128, first = both || turn == 0, second = both || turn == 1;
      if (first)
        ok = mbar_wait_warp(&bars->d_empty[0], (uses0 & 1) ^ 1, abort_flag, status, kSiteDEmpty);
      if (second && ok)
        ok = mbar_wait_warp(&bars->d_empty[1], (uses1 & 1) ^ 1, abort_flag, status, kSiteDEmpty);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem + (first ? 0u : 128u);
      ok = unit_shift<kTwo>(n) == 1
               ? tile_mmas<1, kTwo>(st, bars, xring, tmem, d_tmem, n, a.sbs, abort_flag, status)
               : tile_mmas<2, false>(st, bars, xring, tmem, d_tmem, n, a.sbs, abort_flag, status);
      if (!ok) break;
      if (elect_one()) {
        if (first) commit_pair(&bars->d_full[0]);
        if (second) commit_pair(&bars->d_full[1]);
      }
      __syncwarp();
      uses0 += first, uses1 += second;
      turn = both ? 0 : turn ^ 1;
    }
    if (elect_one()) {
      commit_own(&bars->drain);
      volatile int no_abort = 0;
      mbar_wait_bounded(&bars->drain, 0, &no_abort, status, kSiteDrain);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // ----------------------------------------------------------- dequantise --
    const int me = (warp - 4) / 4, row = 32 * (warp % 4) + lane;
    const uint32_t lanes = (uint32_t)(32 * (warp % 4)) << 16;
    int ws = me, round = 0;  // stage of this group's next super-block
    int gw = 0, unit = 0;  // super-blocks and units of both groups so far
    int last1 = -1, last2 = -1;  // units of this warp's last two halves
    auto scale_of = [&](const Tile& w) {
      return a.scale[((size_t)w.expert * a.bands + band_of(a, w.pair, rank)) * kBand + row];
    };
    float scale = next.n ? scale_of(next) : 1.0f;
    while (next.n && ok) {
      const Tile w = take();
      const bool split = unit_shift<kTwo>(w.n) == 1;  // a unit for each half
      const float inv = 1.0f / fabsf(scale);
      const bool wide = __any_sync(0xffffffffu, scale < 0.0f);
      if (next.n) scale = scale_of(next);
      for (int sb = 0; sb < a.sbs && ok; ++sb, ++gw, unit += split ? 2 : 1) {
        if ((gw & 1) != me) continue;
        if (!(ok = mbar_wait_warp(&bars->w_full[ws], round & 1, abort_flag, status,
                                  kSiteWFull)))
          break;
// (binary16's longer code: 47.3 us rolled up, 48.0 us unrolled, 37.7 GFLOP)
#pragma unroll (__is_same(T, __half) ? 1 : 2)
        for (int h = 0; h < 2; ++h) {
          Half<kFmt> half;
          half.load(wring + ws * kWTile<kFmt>, row, h, inv, wide);
          const int mine = split ? unit + h : unit;
          // in pairs, the same half of each super-block has the same two slots
          const int as = kTwo ? 2 * h : 2 * me + h, last = kTwo ? mine - 2 : last2;
          // The slot's last unit is at most kUnits back, so its barrier has not
          // gone further.
          if (last >= 0 && !(ok = mbar_wait_warp(&bars->done[last % kUnits], (last / kUnits) & 1,
                                                 abort_flag, status, kSiteDone)))
            break;
          last2 = last1, last1 = mine;
          tc_fence_after();
          const uint32_t dst = tmem + lanes + (uint32_t)(kACol0 + as * kACols);
          auto all = [&](auto expand) {
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
              uint32_t v[16];
              expand(cc, v);
              tmem_st16(dst + 16 * cc, v);
            }
          };
          if constexpr (kTwo) {
            all([&](int cc, uint32_t(&v)[16]) {
              uint32_t rest[16];
              half.expand_pair(cc, v, rest);
              tmem_st16(dst + kACols + 16 * cc, rest);
            });
          } else if constexpr (__is_same(T, __half)) {
            all([&](int cc, uint32_t(&v)[16]) { half.expand_once(cc, v); });
          } else if (!wide) {
            all([&](int cc, uint32_t(&v)[16]) { half.template expand<false>(cc, v); });
          } else {
            all([&](int cc, uint32_t(&v)[16]) { half.template expand<true>(cc, v); });
          }
          if (h == 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->w_empty[ws]);
            if ((ws += 2) >= kWStages<kFmt>) ws -= kWStages<kFmt>, ++round;
          }
          if (h == 1 || split) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader_tmem(&bars->ready[mine % kUnits]);
          }
        }
      }
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------- epilogue --
    // Thread (r, c) of a warp, r = lane / 4, holds rows 16 h + r and 16 h + 8 +
    // r of its 32 and items 8 j + 2 c, + 1: pairs of items go to shared memory
    // transposed, [item][row], and from there to Y in 16-byte pieces.
    const int q = warp % 4, me = (warp - 12) / 4;   // me: the accumulator half
    griddep_wait();
    T* Y = static_cast<T*>(a.Y);
    constexpr int kCols = kGlu ? 16 : 32;          // output features of a warp
    constexpr int kPieces = kCols / 8;              // 16-byte units of an item
    constexpr bool kScaled = !__is_same(T, __half);
    constexpr float kUp = kScaled ? 32768.0f : 1.0f;
    uint8_t* stage = out_stage + (warp - 12) * kOutWarp;
    // items of no expert: zeros
    for (long long i = a.offsets[a.E] + (long long)blockIdx.x; i < a.offsets[a.E + 1];
         i += gridDim.x)
      for (int m = 128 * me + 32 * q + lane; m < a.out; m += 256)
        Y[i * a.ldy + m] = from_f32<T>(0.0f);
    int turn = 0, uses = 0;
    while (next.n && ok) {
      const Tile w = take();
      const bool both = w.n > 128, here = both || turn == me;
      turn = both ? 0 : turn ^ 1;
      if (!here) continue;
      const int band = band_of(a, w.pair, rank);
      const bool mine = 2 * w.pair + rank < a.bands;
      const float* sc = a.scale + ((size_t)w.expert * a.bands + band) * kBand + 32 * q + (lane >> 2);
      // (in wide groups of rows the weights are not scaled down further)
      auto up = [&](float s) { return s < 0.0f ? -s : s * kUp; };
      const float scale[4] = {up(sc[0]), up(sc[8]), up(sc[16]), up(sc[24])};
      const int m0 = (band * 4 + q) * kCols;       // this warp's first output feature
      const int item0 = both ? 128 * me : 0;
      const int cols = min(128, w.n - item0), count = mine ? w.count - item0 : 0;
      const uint32_t src = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(128 * me);
      // lane l holds the scales of items l, 32 + l, ...
      float xs[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        xs[k] = kScaled && 32 * k + lane < count ? a.xscale[w.first + item0 + 32 * k + lane] : 1.0f;
      // this lane's first 16-byte unit of a piece, and the step to its next
      constexpr int kStep = 32 / kPieces;
      const int item = lane / kPieces, unit = lane % kPieces, m = m0 + 8 * unit;
      T* y = Y + (w.first + item0 + item) * a.ldy + m;
      const long long step = (long long)kStep * a.ldy;
      const bool whole = a.vec && m + 8 <= a.out;
      if (!(ok = mbar_wait_warp(&bars->d_full[me], uses & 1, abort_flag, status, kSiteDFull))) break;
      ++uses;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c0 = 32 * k;
        if (c0 >= cols) break;
        uint32_t v[2][16];
        tmem_ld_frag(src + c0, v[0]);
        tmem_ld_frag(src + c0 + (16u << 16), v[1]);
        tmem_wait_frag(v[0], v[1]);
        if (c0 + 32 >= cols) {  // the accumulator is in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_leader_tmem(&bars->d_empty[me]);
        }
        uint32_t p[4][4];  // [j][unit]: item pairs of 8-row blocks
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x0 = kScaled ? __shfl_sync(0xffffffffu, xs[k], 8 * j + 2 * (lane & 3)) : 1.0f;
          const float x1 =
              kScaled ? __shfl_sync(0xffffffffu, xs[k], 8 * j + 2 * (lane & 3) + 1) : 1.0f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              f[e] = __uint_as_float(v[h][4 * j + e]) * scale[2 * h + e / 2] * (e % 2 ? x1 : x0);
            if constexpr (kGlu) {
              p[j][h] = pack2<T>(silu(f[0]) * f[2], silu(f[1]) * f[3]);
            } else {
              p[j][2 * h] = pack2<T>(f[0], f[1]);
              p[j][2 * h + 1] = pack2<T>(f[2], f[3]);
            }
          }
        }
        __syncwarp();  // the last piece has left the staging
        if constexpr (kGlu) {
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const int i = 8 * (j + (lane >> 4)) + (lane & 7), u = (lane >> 3) & 1;
            store_tiles_t(smem_u32(stage + i * 32 + (u ^ ((i >> 2) & 1)) * 16), p[j][0], p[j][1],
                          p[j + 1][0], p[j + 1][1]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = 8 * j + (lane & 7), u = lane >> 3;
            store_tiles_t(smem_u32(stage + i * 64 + (u ^ ((i >> 1) & 3)) * 16), p[j][0], p[j][1],
                          p[j][2], p[j][3]);
          }
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < kPieces; ++r, y += step) {
          const int i = item + kStep * r;
          const int at = kGlu ? unit ^ ((i >> 2) & 1) : unit ^ ((i >> 1) & 3);
          const uint4 u = *reinterpret_cast<const uint4*>(stage + (i * kPieces + at) * 16);
          if (c0 + i >= count) continue;
          if (whole) {
            *reinterpret_cast<uint4*>(y) = u;
          } else {
            const T* one = reinterpret_cast<const T*>(&u);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (m + e < a.out) y[e] = one[e];
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other may still signal it
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

typedef void (*Kernel)(const RowMaps, const Args, unsigned int*);
template <typename T>
Kernel pick_t(int fmt, int swiglu) {
  if (fmt == Q6_FMT_Q4K)
    return swiglu ? experts_tc_kernel<T, Q6_FMT_Q4K, true> : experts_tc_kernel<T, Q6_FMT_Q4K, false>;
  return swiglu ? experts_tc_kernel<T, Q6_FMT_Q6K, true> : experts_tc_kernel<T, Q6_FMT_Q6K, false>;
}
Kernel pick(int type, int fmt, int swiglu) {
  return type == Q6_TYPE_BF16 ? pick_t<__nv_bfloat16>(fmt, swiglu) : pick_t<__half>(fmt, swiglu);
}
int smem_bytes(int fmt) {
  return fmt == Q6_FMT_Q4K ? kSmemBytes<Q6_FMT_Q4K> : kSmemBytes<Q6_FMT_Q6K>;
}
static_assert(kSmemBytes<Q6_FMT_Q4K> <= 227 * 1024 && kSmemBytes<Q6_FMT_Q6K> <= 227 * 1024,
              "shared memory");

// Fills a launch of `pairs` CTA pairs; attr holds two attributes.
void pair_launch(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int fmt, unsigned pairs,
                 cudaStream_t s) {
  *cfg = cudaLaunchConfig_t{};
  cfg->gridDim = dim3(2 * pairs);
  cfg->blockDim = dim3(kThreads);
  cfg->dynamicSmemBytes = (size_t)smem_bytes(fmt);
  cfg->stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 2;
}

// CTA pairs each device runs at a time (a device's SMs need not all pair up).
int g_pairs[64];

}  // namespace

cudaError_t experts_tc_prepare() {
  int dev = 0, least = 1 << 30;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  for (int type : {Q6_TYPE_BF16, Q6_TYPE_F16})
    for (int fmt : {Q6_FMT_Q4K, Q6_FMT_Q6K})
      for (int glu : {0, 1}) {
        const Kernel k = pick(type, fmt, glu);
        if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      smem_bytes(fmt))) != cudaSuccess)
          return e;
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        pair_launch(&cfg, attr, fmt, 1, nullptr);
        cfg.numAttrs = 1;
        int n = 0;
        if ((e = cudaOccupancyMaxActiveClusters(&n, k, &cfg)) != cudaSuccess) return e;
        least = n < least ? n : least;
      }
  if (least < 1) return cudaErrorInvalidConfiguration;
  g_pairs[dev % 64] = least;
  return cudaSuccess;
}

cudaError_t launch_experts_tc(const ExpertCall& c, const RowMaps& x, const float* scale,
                              bool x_made, unsigned int* status, cudaStream_t s) {
  Args a;
  a.plane = c.plane;
  a.scale = reinterpret_cast<const float*>(c.plane + c.g.scale_off);
  a.xscale = scale;
  a.offsets = c.offsets;
  a.Y = c.Y, a.ldy = c.ldy;
  a.E = c.E, a.bands = c.g.bands, a.sbs = c.g.sbs, a.out = c.g.out;
  a.vec = (reinterpret_cast<uintptr_t>(c.Y) | (uintptr_t)(c.ldy * 2)) % 16 == 0;
  a.early = x_made;
  // at most this many tiles
  const long long tiles =
      (c.items / kTileN + (c.items < c.E ? c.items : c.E) + 1) * (long long)((c.g.bands + 1) / 2);
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const long long most = g_pairs[dev % 64];
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  pair_launch(&cfg, attr, c.fmt, (unsigned)(tiles < most ? tiles : most), s);
  return cudaLaunchKernelEx(&cfg, pick(c.type, c.fmt, c.swiglu), x, a, status);
}

// ------------------------------------------------------- x in item order ---
namespace {
constexpr int kRowThreads = 128;
// One block an item: xh[i] = its row of X as binary16, bf16 rows times 2^-e
// with the largest finite value in [2^14, 2^15), and scale[i] = 2^e.
template <typename T>
__global__ void __launch_bounds__(kRowThreads)
expert_rows_kernel(const T* X, long long ldx, const int32_t* rows, int units, uint4* xh,
                   float* scale) {
  constexpr int kKeep = 4;  // units a thread keeps in registers; longer rows are read again
  __shared__ uint32_t part[kRowThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const long long i = blockIdx.x;
  const uint4* src = reinterpret_cast<const uint4*>(X + (rows ? rows[i] : i) * ldx);
  uint4* dst = xh + i * units;
  uint4 v[kKeep];
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int u = threadIdx.x + kRowThreads * k;
    v[k] = u < units ? src[u] : make_uint4(0, 0, 0, 0);
  }
  if constexpr (__is_same(T, __half)) {
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
      if (threadIdx.x + kRowThreads * k < units) dst[threadIdx.x + kRowThreads * k] = v[k];
    for (int u = threadIdx.x + kRowThreads * kKeep; u < units; u += kRowThreads) dst[u] = src[u];
  } else {
    uint32_t most = 0;  // of the values' bits without the sign, infinities and NaN left out
    auto size = [&](const uint4& u) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w = word4(u, k) & 0x7FFF7FFFu, lo = w & 0xFFFFu, hi = w >> 16;
        if (lo < 0x7F80u) most = max(most, lo);
        if (hi < 0x7F80u) most = max(most, hi);
      }
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k) size(v[k]);
    for (int u = threadIdx.x + kRowThreads * kKeep; u < units; u += kRowThreads) size(src[u]);
    most = __reduce_max_sync(0xffffffffu, most);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = most;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kRowThreads / 32; ++k) most = max(most, part[k]);
    // 2^e and 2^-e normal numbers
    const int e = min(max((int)(most >> 7) - 127 - 14, -116), 118);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    auto half = [&](const uint4& u) {
      uint32_t h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = unpack2<T>(word4(u, k));
        h[k] = pack2<__half>(f.x * down, f.y * down);
      }
      return make_uint4(h[0], h[1], h[2], h[3]);
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
      if (threadIdx.x + kRowThreads * k < units) dst[threadIdx.x + kRowThreads * k] = half(v[k]);
    for (int u = threadIdx.x + kRowThreads * kKeep; u < units; u += kRowThreads)
      dst[u] = half(src[u]);
    if (threadIdx.x == 0) scale[i] = __uint_as_float((uint32_t)(127 + e) << 23);
  }
}
}  // namespace

cudaError_t launch_expert_rows(const ExpertCall& c, int K, __half* xh, float* scale,
                               cudaStream_t s) {
  const int32_t* rows = c.gather ? c.rows : nullptr;
  const dim3 grid((unsigned)c.items);
  uint4* out = reinterpret_cast<uint4*>(xh);
  return c.type == Q6_TYPE_BF16
             ? launch_pdl(expert_rows_kernel<__nv_bfloat16>, grid, dim3(kRowThreads), 0, s,
                          static_cast<const __nv_bfloat16*>(c.X), c.ldx, rows, K / 8, out, scale)
             : launch_pdl(expert_rows_kernel<__half>, grid, dim3(kRowThreads), 0, s,
                          static_cast<const __half*>(c.X), c.ldx, rows, K / 8, out, scale);
}

}  // namespace q6
