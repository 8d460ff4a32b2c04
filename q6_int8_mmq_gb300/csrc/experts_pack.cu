// Packing of raw K-quant expert matrices into the expert plane (its layout is
// described in moe_internal.cuh). Load time: one block per tile, the raw
// blocks of its 128 rows staged in shared memory, then one thread a row.
#include "moe_internal.cuh"

namespace q6 {
namespace {

constexpr int kQ4Raw = 144, kQ6Raw = 210;

// The raw row behind plane row p of an expert, or -1 for padding.
__device__ __forceinline__ int raw_row(int p, int M, int swiglu) {
  if (!swiglu) return p < M ? p : -1;
  const int o = p / 16 * 8 + p % 8;
  if (o >= M / 2) return -1;
  return (p % 16 < 8 ? 0 : M / 2) + o;
}

template <int kRaw>
__global__ void __launch_bounds__(kBand)
expert_pack_kernel(const uint8_t* raw, int M, int swiglu, int bands, int sbs, uint8_t* plane) {
  constexpr int kTile = kRaw == kQ4Raw ? kQ4Tile : kQ6Tile;
  constexpr int kPitch = ((kRaw + 3) / 4 | 1) * 4;  // odd multiple of 4 bytes
  __shared__ uint8_t blk[kBand * kPitch];
  const size_t tile = blockIdx.x;  // [expert][band][super-block]
  const int sb = (int)(tile % sbs);
  const int band = (int)(tile / sbs % bands);
  const size_t e = tile / sbs / bands;
  for (int i = threadIdx.x; i < kBand * kRaw; i += kBand) {
    const int r = raw_row(band * kBand + i / kRaw, M, swiglu);
    blk[i / kRaw * kPitch + i % kRaw] =
        r < 0 ? 0 : raw[((e * M + r) * sbs + sb) * (size_t)kRaw + i % kRaw];
  }
  __syncthreads();
  const int row = threadIdx.x;
  const uint8_t* b = blk + row * kPitch;
  uint4* out = reinterpret_cast<uint4*>(plane + tile * kTile) + row;
  auto unit = [&](int u, const uint32_t (&w)[4]) {
    out[u * kBand] = make_uint4(w[0], w[1], w[2], w[3]);
  };
  // code of element k of the row's block: 4 or 6 bits
  auto code = [&](int k) -> uint32_t {
    if (kRaw == kQ4Raw) {
      const int sub = k / 32;
      return (b[16 + 32 * (sub / 2) + k % 32] >> (4 * (sub % 2))) & 15u;
    }
    const int h = k / 128, r = k % 128;
    const uint32_t lo = (b[64 * h + r % 64] >> (4 * (r / 64))) & 15u;
    return lo | ((b[128 + 32 * h + r % 32] >> (2 * (r / 32))) & 3u) << 4;
  };
  if (kRaw == kQ4Raw) {
    uint32_t w[4];
    for (int i = 0; i < 4; ++i)
      w[i] = b[4 * i] | (uint32_t)b[4 * i + 1] << 8 | (uint32_t)b[4 * i + 2] << 16 |
             (uint32_t)b[4 * i + 3] << 24;
    unit(0, w);
  }
  for (int j = 0; j < 8; ++j) {
    uint32_t w[4];
    for (int cc = 0; cc < 4; ++cc) {
      const int k0 = 32 * (4 * (j % 2) + cc) + 8 * (j / 2);
      w[cc] = 0;
      for (int i = 0; i < 8; ++i) w[cc] |= (code(k0 + i) & 15u) << (4 * (i / 2 + 4 * (i % 2)));
    }
    unit((kRaw == kQ4Raw ? 1 : 0) + j, w);
  }
  if (kRaw == kQ6Raw) {
    for (int t = 0; t < 4; ++t) {
      uint32_t w[4] = {};
      for (int c = 0; c < 8; ++c)
        for (int i = 0; i < 8; ++i)
          w[c / 2] |= (code(32 * c + 8 * t + i) >> 4) << (4 * (i / 2) + 2 * (c % 2) + 16 * (i % 2));
      unit(8 + t, w);
    }
    uint32_t w[4] = {};
    for (int i = 0; i < 16; ++i) {
      const int at = (i % 2) * 8 + i / 2;
      w[at / 4] |= (uint32_t)(b[192 + i] ^ 0x80u) << (8 * (at % 4));
    }
    unit(12, w);
    uint16_t* d = reinterpret_cast<uint16_t*>(plane + tile * kTile + 13 * 2048);
    d[row] = (uint16_t)(b[208] | b[209] << 8);
  }
}

// 2^e of each plane row, from an upper bound of its weights' size; negative for 32
// rows of which one has a super-block whose bound is below kWideRange of the row's
// (and not 0).
constexpr float kWideRange = 1.0f / 128.0f;
template <int kRaw>
__global__ void __launch_bounds__(kBand)
expert_scale_kernel(const uint8_t* plane, int sbs, float* scale) {
  constexpr int kTile = kRaw == kQ4Raw ? kQ4Tile : kQ6Tile;
  const size_t band = blockIdx.x;
  const int row = threadIdx.x;
  float most = 0.0f, least = INFINITY;
  for (int sb = 0; sb < sbs; ++sb) {
    const uint8_t* t = plane + (band * sbs + sb) * kTile;
    float v;
    if (kRaw == kQ4Raw) {
      const __half* d = reinterpret_cast<const __half*>(t + row * 16);
      v = 63.0f * 15.0f * fabsf(__half2float(d[0])) + 63.0f * fabsf(__half2float(d[1]));
    } else {
      v = 128.0f * 32.0f *
          fabsf(__half2float(reinterpret_cast<const __half*>(t + 13 * 2048)[row]));
    }
    if (!(v < 1e30f)) continue;  // an infinite or NaN scale shows whatever e is
    most = fmaxf(most, v);
    if (v > 0.0f) least = fminf(least, v);
  }
  const float s = most > 0.0f ? ldexpf(1.0f, ilogbf(most) + 1 - 10) : 1.0f;
  const bool wide = __any_sync(0xffffffffu, least < most * kWideRange);
  scale[band * kBand + row] = wide ? -s : s;
}

template <int kRaw>
cudaError_t pack(const uint8_t* raw, int E, int M, int swiglu, const ExpertGeom& g, uint8_t* plane,
                 cudaStream_t s) {
  const unsigned bands = (unsigned)E * (unsigned)g.bands;
  expert_pack_kernel<kRaw><<<bands * (unsigned)g.sbs, kBand, 0, s>>>(raw, M, swiglu, g.bands,
                                                                     g.sbs, plane);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  expert_scale_kernel<kRaw><<<bands, kBand, 0, s>>>(
      plane, g.sbs, reinterpret_cast<float*>(plane + g.scale_off));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_pack(int fmt, const uint8_t* raw, int E, int M, int K, int swiglu,
                               uint8_t* plane, cudaStream_t s) {
  const ExpertGeom g = expert_geom(fmt, E, M, K, swiglu);
  return fmt == Q6_FMT_Q4K ? pack<kQ4Raw>(raw, E, M, swiglu, g, plane, s)
                           : pack<kQ6Raw>(raw, E, M, swiglu, g, plane, s);
}

}  // namespace q6
