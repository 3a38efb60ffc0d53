// 4-bit weights (E2M1 codes, one power of two a group of 32; layout in fp4.h):
// from float weights, from a checkpoint's row-major codes, and back to values.
//
// The scale of a group is the smallest 2^e with max|v| / 6 <= 2^e (6: the
// largest code's value), e >= -125, read from the bits of max|v|; v / 2^e is
// exact, so a code is one rounding of the weight itself (nearest, ties to even)
// and every value it stands for is a normal bf16 number or zero.  No largest
// value is clipped; only from 1.75 2^127 on, where the nearest value would be
// 2^128, the code below it is taken.  A group with an element that is not finite
// gets the NaN scale and zero codes.
//
// A wave makes four tiles of 16 rows along K: the lane of row r and group g
// reads its 32 weights of each, and writes 16 bytes of codes a tile and one dword
// of four scales.
#include "common.h"
#include "fp4.h"
#include "kernels.h"
#include "ops.h"

namespace moelora {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr uint32_t kInfBits = 0x7f800000u;

// Which four tiles (a "quad") a wave makes, and its lane's place in them.
struct Quad {
  uint32_t tile_row, q;  // of all matrices; along K
  int n, k0, g;        // row in the matrix; column of its group in the first tile
  bool some;           // the row exists
};
__device__ __forceinline__ Quad quad_of(const Fp4WeightsArgs &a) {
  const int lane = threadIdx.x % kWave;
  const uint32_t id = blockIdx.x * kWaves + threadIdx.x / kWave;  // (fewer than 2^26)
  Quad q;
  q.tile_row = id / a.KQ;
  q.q = id % a.KQ;
  q.g = lane / kTileRows;
  q.n = (int)(q.tile_row % a.NT) * kTileRows + lane % kTileRows;
  q.k0 = (int)q.q * 4 * kTileCols + q.g * kGroup;
  q.some = q.n < a.N;
  return q;
}
__device__ __forceinline__ bool quad_exists(const Fp4WeightsArgs &a) {
  return blockIdx.x * kWaves + threadIdx.x / kWave < (uint32_t)a.mats * a.NT * a.KQ;
}
__device__ __forceinline__ uint4 *tile_codes(uint8_t *codes, const Fp4WeightsArgs &a, const Quad &q, int b) {
  return reinterpret_cast<uint4 *>(codes + ((size_t)q.tile_row * a.KB + q.q * 4 + b) * kTileBytes) + threadIdx.x % kWave;
}
__device__ __forceinline__ uint32_t *quad_scales(uint8_t *scales, const Fp4WeightsArgs &a, const Quad &q) {
  return reinterpret_cast<uint32_t *>(scales + ((size_t)q.tile_row * a.KQ + q.q) * kScaleBytes) + threadIdx.x % kWave;
}

// 32 elements of a row of K from element c on, zeros past K, as float32.
template <typename DT>
__device__ __forceinline__ void load32(const DT *row, int c, int K, bool some, float *f) {
  typedef u32x4_t mem __attribute__((aligned(2)));
  constexpr int n = sizeof(DT) * 2, per = 16 / sizeof(DT);
  if (some && c + kGroup <= K) {
    const mem *p = reinterpret_cast<const mem *>(row + c);
    u32x4_t v[n];
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = p[i];
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const Chunk<DT> e = chunk_elems<DT>(v[i]);
#pragma unroll
      for (int j = 0; j < per; ++j) f[per * i + j] = Elem<DT>::to_f32(e.v[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kGroup; ++i) f[i] = some && c + i < K ? Elem<DT>::to_f32(row[c + i]) : 0.f;
  }
}

template <typename DT>
__global__ __launch_bounds__(kThreads) void k_quant_fp4(Fp4WeightsArgs a) {
  if (!quad_exists(a)) return;
  const Quad q = quad_of(a);
  const DT *row = static_cast<const DT *>(a.src) + ((size_t)(q.tile_row / a.NT) * a.N + q.n) * a.K;
  uint32_t scales = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    if (q.q * 4 + b >= (uint32_t)a.KB) break;
    float f[kGroup];
    load32<DT>(row, q.k0 + b * kTileCols, a.K, q.some, f);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
    // amax = (1 + f) 2^q: amax / 6 <= 2^(q - 2) exactly when 1 + f <= 1.5
    const int e = max(-125, (int)(m >> 23) - 127 - 2 + ((m & 0x7fffffu) > 0x400000u));
    const bool odd = m >= kInfBits;
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    uint32_t c[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      uint32_t w = 0;
#define MOELORA_PAIR(s) \
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[8 * d + 2 * s] * inv, f[8 * d + 2 * s + 1] * inv, 1.f, s)
      MOELORA_PAIR(0);
      MOELORA_PAIR(1);
      MOELORA_PAIR(2);
      MOELORA_PAIR(3);
#undef MOELORA_PAIR
      if (e == 126) {  // 4 2^126 is not finite: 3 2^126 then (codes 6, 14 -> 5, 13)
        const uint32_t six = w >> 1 & w >> 2 & ~w & 0x11111111u;
        w -= six;
      }
      c[d] = odd ? 0u : w;
    }
    *tile_codes(a.codes, a, q, b) = make_uint4(c[0], c[1], c[2], c[3]);
    scales |= (odd ? 255u : q.some && q.k0 + b * kTileCols < a.K ? (uint32_t)(e + 127) : 0u) << 8 * b;
  }
  *quad_scales(a.scales, a, q) = scales;
}

// Row-major codes, two a byte and ceil(K / 2) bytes a row, with ceil(K / 32) scales.
__global__ __launch_bounds__(kThreads) void k_pack_fp4(Fp4WeightsArgs a) {
  if (!quad_exists(a)) return;
  const Quad q = quad_of(a);
  const int row_bytes = (a.K + 1) / 2, row_groups = (a.K + kGroup - 1) / kGroup;
  const size_t r = (size_t)(q.tile_row / a.NT) * a.N + q.n;
  const uint8_t *row = static_cast<const uint8_t *>(a.src) + r * row_bytes;
  const uint8_t *rs = a.src_scales + r * row_groups;
  typedef u32x4_t mem __attribute__((aligned(1)));
  uint32_t scales = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    if (q.q * 4 + b >= (uint32_t)a.KB) break;
    const int k = q.k0 + b * kTileCols, at = k / 2;
    u32x4_t c = {0, 0, 0, 0};
    if (q.some && k + kGroup <= a.K) {
      c = *reinterpret_cast<const mem *>(row + at);
    } else if (q.some && k < a.K) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        uint32_t v = k + 2 * i < a.K ? row[at + i] : 0u;
        if (k + 2 * i + 1 >= a.K) v &= 15u;
        c[i / 4] |= v << 8 * (i % 4);
      }
    }
    if (q.some && k < a.K) scales |= (uint32_t)rs[k / kGroup] << 8 * b;
    *tile_codes(a.codes, a, q, b) = __builtin_bit_cast(uint4, c);
  }
  *quad_scales(a.scales, a, q) = scales;
}

template <typename DT>
__global__ __launch_bounds__(kThreads) void k_dequant_fp4(Fp4WeightsArgs a) {
  if (!quad_exists(a)) return;
  const Quad q = quad_of(a);
  const uint32_t scales = *quad_scales(a.scales, a, q);
  DT *row = static_cast<DT *>(a.dst) + ((size_t)(q.tile_row / a.NT) * a.N + q.n) * a.K;
  typedef u32x4_t mem __attribute__((aligned(2)));
  constexpr int per = 16 / sizeof(DT);
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int k = q.k0 + b * kTileCols;
    if (!q.some || k >= a.K) break;
    const uint4 c = *tile_codes(a.codes, a, q, b);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    const float s = scale_of_code(scales >> 8 * b & 255u);
    u32x4_t v[32 / per];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if constexpr (sizeof(DT) == 2) {
        v[d] = e2m1x8_to_bf16(w[d], s);
      } else {
        typedef float f32x2_t __attribute__((ext_vector_type(2)));
        const f32x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[d], s, 0),
                      p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[d], s, 1),
                      p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[d], s, 2),
                      p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[d], s, 3);
        v[2 * d] = __builtin_bit_cast(u32x4_t, f32x4_t{p0[0], p0[1], p1[0], p1[1]});
        v[2 * d + 1] = __builtin_bit_cast(u32x4_t, f32x4_t{p2[0], p2[1], p3[0], p3[1]});
      }
    }
#pragma unroll
    for (int i = 0; i < 32 / per; ++i) {
      if (k + (i + 1) * per <= a.K) {
        *reinterpret_cast<mem *>(row + k + i * per) = v[i];
      } else {
        const Chunk<DT> e = chunk_elems<DT>(v[i]);
#pragma unroll
        for (int j = 0; j < per; ++j)
          if (k + i * per + j < a.K) row[k + i * per + j] = e.v[j];
      }
    }
  }
}

template <typename K>
hipError_t launch(K kern, const Fp4WeightsArgs &a, hipStream_t st) {
  const size_t quads = (size_t)a.mats * a.NT * a.KQ;
  return launch_kernel(kern, dim3((unsigned)((quads + kWaves - 1) / kWaves)), dim3(kThreads), 0, st, a);
}

}  // namespace

hipError_t launch_quantize_fp4(const Fp4WeightsArgs &a, bool bf16, hipStream_t st) {
  return bf16 ? launch(k_quant_fp4<uint16_t>, a, st) : launch(k_quant_fp4<float>, a, st);
}

hipError_t launch_pack_fp4(const Fp4WeightsArgs &a, hipStream_t st) { return launch(k_pack_fp4, a, st); }

hipError_t launch_dequantize_fp4(const Fp4WeightsArgs &a, bool bf16, hipStream_t st) {
  return bf16 ? launch(k_dequant_fp4<uint16_t>, a, st) : launch(k_dequant_fp4<float>, a, st);
}

}  // namespace moelora
