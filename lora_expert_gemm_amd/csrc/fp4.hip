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
// A wave makes four tiles of 16 rows along K, "a quad".  On the side of the rows its
// lanes lie along them, 16 bytes each, so that whole lines move; what a group's lanes hold
// (4 of 8 bf16 elements, 8 of 4 float32 ones) meets in one entry of the tile.
//
// Bound by HBM: 16 x 11008 x 4096 bf16 made into codes in 302 us (6.0 TB/s, mostly read)
// and back in 357 (5.1 TB/s, mostly written; a large copy 5.0).
#include "common.h"
#include "fp4.h"
#include "kernels.h"
#include "ops.h"

namespace moelora {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr uint32_t kInfBits = 0x7f800000u;

// Which quad a wave makes.
struct Quad {
  uint32_t tile_row, q;  // of all matrices; along K
  int n0, k0, mat;       // first row in its matrix, first column
};
__device__ __forceinline__ bool quad_of(const Fp4WeightsArgs &a, Quad &q) {
  const uint32_t id = __builtin_amdgcn_readfirstlane(blockIdx.x * kWaves + threadIdx.x / kWave);  // (below 2^26)
  q.tile_row = id / a.KQ;
  q.q = id % a.KQ;
  q.mat = q.tile_row / a.NT;
  q.n0 = (int)(q.tile_row % a.NT) * kTileRows;
  q.k0 = (int)q.q * 4 * kTileCols;
  return id < (uint32_t)a.mats * a.NT * a.KQ;
}
__device__ __forceinline__ uint8_t *tile_codes(const Fp4WeightsArgs &a, const Quad &q, int b) {
  return a.codes + ((size_t)q.tile_row * a.KB + q.q * 4 + b) * kTileBytes;
}
__device__ __forceinline__ uint32_t *quad_scales(const Fp4WeightsArgs &a, const Quad &q) {
  return reinterpret_cast<uint32_t *>(a.scales + ((size_t)q.tile_row * a.KQ + q.q) * kScaleBytes);
}

// How a wave's lanes lie on a tile's rows: PER elements (16 bytes) each, LANES a
// row, ROWS rows at a time, STEPS times.
template <typename DT> struct Lanes {
  static constexpr int PER = 16 / (int)sizeof(DT), LANES = kTileCols / PER, ROWS = kWave / LANES,
                       STEPS = kTileRows / ROWS, GROUP = kGroup / PER;  // lanes a group
  int r, c;  // row of the step, lane of the row
  __device__ __forceinline__ Lanes() : r(threadIdx.x % kWave / LANES), c(threadIdx.x % LANES) {}
  __device__ __forceinline__ int row(int s) const { return s * ROWS + r; }
  // the lane's entry in the tile, and its bytes in there (half a byte an element)
  __device__ __forceinline__ int entry(int s) const { return c / GROUP * kTileRows + row(s); }
  __device__ __forceinline__ int byte(int s) const { return entry(s) * 16 + c % GROUP * (PER / 2); }
};
// WHOLE: rows of whole lines pass by the caches; of others, a line's two owners meet there (16 x
// 11008 x 4090 bf16 quantised 358 us, past the caches 476; 4096 columns, quantised and back in turn,
// past the caches 656, through them 690).
template <typename DT> bool whole_lines(int K) { return K % (128 / (int)sizeof(DT)) == 0; }
template <int BYTES> struct CodeWord;
template <> struct CodeWord<4> { typedef uint32_t type; };
template <> struct CodeWord<2> { typedef uint16_t type; };

template <bool WHOLE, typename DT>
__global__ __launch_bounds__(kThreads) void k_quant_fp4(Fp4WeightsArgs a) {
  typedef Lanes<DT> L;
  typedef typename CodeWord<L::PER / 2>::type word;
  typedef u32x4_t mem __attribute__((aligned(2)));
  Quad q;
  if (!quad_of(a, q)) return;
  const L ln;
  const DT *const w = static_cast<const DT *>(a.src) + ((size_t)q.mat * a.N + q.n0) * a.K;
  const int rows = min(kTileRows, a.N - q.n0);
  uint32_t scales[L::STEPS];
#pragma unroll
  for (int s = 0; s < L::STEPS; ++s) scales[s] = 0;
  const int tiles = min(4, a.KB - (int)q.q * 4);
  for (int b = 0; b < tiles; ++b) {
    const int k = q.k0 + b * kTileCols + ln.c * L::PER;
    u32x4_t v[L::STEPS];
#pragma unroll
    for (int s = 0; s < L::STEPS; ++s) {
      const DT *row = w + (size_t)min(ln.row(s), rows - 1) * a.K;
      if (k + L::PER <= a.K) {
        const mem *p = reinterpret_cast<const mem *>(row + k);
        if constexpr (WHOLE) v[s] = __builtin_nontemporal_load(p);
        else v[s] = *p;
      } else {
        Chunk<DT> e;
#pragma unroll
        for (int i = 0; i < L::PER; ++i) e.v[i] = k + i < a.K ? row[k + i] : DT(0);
        v[s] = __builtin_bit_cast(u32x4_t, e);
      }
    }
    uint8_t *const tile = tile_codes(a, q, b);
#pragma unroll
    for (int s = 0; s < L::STEPS; ++s) {
      const Chunk<DT> e = chunk_elems<DT>(v[s]);
      const bool some = ln.row(s) < rows;
      float f[L::PER];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < L::PER; ++i) {
        f[i] = some ? Elem<DT>::to_f32(e.v[i]) : 0.f;
        m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
      }
#pragma unroll
      for (int d = 1; d < L::GROUP; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
      // amax = (1 + f) 2^x: amax / 6 <= 2^(x - 2) exactly when 1 + f <= 1.5
      const int x = max(-125, (int)(m >> 23) - 127 - 2 + ((m & 0x7fffffu) > 0x400000u));
      const bool odd = m >= kInfBits;
      const float inv = __uint_as_float((uint32_t)(127 - x) << 23);
      uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, f[0] * inv, f[1] * inv, 1.f, 0);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[2] * inv, f[3] * inv, 1.f, 1);
      if constexpr (L::PER == 8) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[4] * inv, f[5] * inv, 1.f, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[6] * inv, f[7] * inv, 1.f, 3);
      }
      if (x == 126) c -= c >> 1 & c >> 2 & ~c & 0x11111111u;  // 4 2^126 is not finite: codes 6, 14 -> 5, 13
      if (odd) c = 0;
      *reinterpret_cast<word *>(tile + ln.byte(s)) = (word)c;
      scales[s] |= (odd ? 255u : some && k / kGroup * kGroup < a.K ? (uint32_t)(x + 127) : 0u) << 8 * b;
    }
  }
  if (ln.c % L::GROUP == 0) {
#pragma unroll
    for (int s = 0; s < L::STEPS; ++s) quad_scales(a, q)[ln.entry(s)] = scales[s];
  }
}

// Row-major codes, two a byte and ceil(K / 2) bytes a row, with ceil(K / 32) scales:
// a group of codes is an entry of a tile as it is.
__global__ __launch_bounds__(kThreads) void k_pack_fp4(Fp4WeightsArgs a) {
  typedef u32x4_t mem __attribute__((aligned(1)));
  Quad q;
  if (!quad_of(a, q)) return;
  const int lane = threadIdx.x % kWave, rows = min(kTileRows, a.N - q.n0);
  const int row_bytes = (a.K + 1) / 2, row_groups = (a.K + kGroup - 1) / kGroup;
  const size_t r0 = (size_t)q.mat * a.N + q.n0;
  {
    // a lane's row and group, of each of the four tiles
    const int r = lane % kTileRows, g0 = q.k0 / kGroup + lane / kTileRows;
    const uint8_t *rs = a.src_scales + (r0 + min(r, rows - 1)) * row_groups;
    uint32_t s = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b)
      s |= (r < rows && g0 + 4 * b < row_groups ? (uint32_t)rs[min(g0 + 4 * b, row_groups - 1)] : 0u) << 8 * b;
    quad_scales(a, q)[lane] = s;
  }
  // 16 groups of a row side by side, four rows at a time
  const int b = lane % 16 / 4, k = q.k0 + lane % 16 * kGroup, at = k / 2;
  u32x4_t c[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int r = 4 * s + lane / 16;
    const uint8_t *row = static_cast<const uint8_t *>(a.src) + (r0 + min(r, rows - 1)) * row_bytes;
    c[s] = u32x4_t{0, 0, 0, 0};
    if (r < rows && k + kGroup <= a.K) {
      c[s] = *reinterpret_cast<const mem *>(row + at);
    } else if (r < rows && k < a.K) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        uint32_t v = k + 2 * i < a.K ? row[at + i] : 0u;
        if (k + 2 * i + 1 >= a.K) v &= 15u;
        c[s][i / 4] |= v << 8 * (i % 4);
      }
    }
  }
  if (q.q * 4 + b >= (uint32_t)a.KB) return;
  uint4 *const tile = reinterpret_cast<uint4 *>(tile_codes(a, q, b));
#pragma unroll
  for (int s = 0; s < 4; ++s)
    tile[lane % 4 * kTileRows + 4 * s + lane / 16] = __builtin_bit_cast(uint4, c[s]);
}

// A quad's values, the lanes on ROWS rows at a time.
template <int ROWS, bool WHOLE, typename DT>
__device__ __forceinline__ void dequant_quad(const Fp4WeightsArgs &a, const Quad &q, uint32_t scales, int width) {
  constexpr int PER = 16 / (int)sizeof(DT), LANES = kWave / ROWS;
  typedef typename CodeWord<PER / 2>::type word;
  typedef u32x4_t mem __attribute__((aligned(2)));
  const int lane = threadIdx.x % kWave, rows = min(kTileRows, a.N - q.n0), r0 = lane / LANES;
  DT *const w = static_cast<DT *>(a.dst) + ((size_t)q.mat * a.N + q.n0) * a.K;
  for (int l0 = 0; l0 < width; l0 += LANES) {
    const int col = (l0 + lane % LANES) * PER, k = q.k0 + col;
    const int b = min(col / kTileCols, a.KB - 1 - (int)q.q * 4), g = col % kTileCols / kGroup;
    const uint8_t *const codes = tile_codes(a, q, b) + (g * kTileRows + r0) * 16 + col % kGroup / 2;
    uint32_t c[kTileRows / ROWS];
#pragma unroll
    for (int i = 0; i < kTileRows / ROWS; ++i) c[i] = *reinterpret_cast<const word *>(codes + i * ROWS * 16);
#pragma unroll
    for (int i = 0; i < kTileRows / ROWS; ++i) {
      const int r = i * ROWS + r0;
      const float sc = scale_of_code((uint32_t)__shfl((int)scales, g * kTileRows + r) >> 8 * b & 255u);
      u32x4_t v;
      if constexpr (sizeof(DT) == 2) {
        v = e2m1x8_to_bf16(c[i], sc);
      } else {
        typedef float f32x2_t __attribute__((ext_vector_type(2)));
        const f32x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], sc, 0),
                      hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], sc, 1);
        v = __builtin_bit_cast(u32x4_t, f32x4_t{lo[0], lo[1], hi[0], hi[1]});
      }
      if (r < rows) {
        DT *const row = w + (size_t)r * a.K;
        if (k + PER <= a.K) {
          mem *const p = reinterpret_cast<mem *>(row + k);
          if constexpr (WHOLE) __builtin_nontemporal_store(v, p);
          else *p = v;
        } else {
          const Chunk<DT> e = chunk_elems<DT>(v);
#pragma unroll
          for (int n = 0; n < PER; ++n)
            if (k + n < a.K) row[k + n] = e.v[n];
        }
      }
    }
  }
}

// A row at a time, so that a store is 1 KB of it: of rows that are no whole lines only the
// first and last line of those are shared (16 x 11008 x 4090 bf16 400 us, by stores of 256 bytes
// of four rows 633).  Two or four rows where a quad has few columns (44 x 3572 x 68 bf16 9 us, a
// row at a time 17).
template <bool WHOLE, typename DT>
__global__ __launch_bounds__(kThreads) void k_dequant_fp4(Fp4WeightsArgs a) {
  constexpr int PER = 16 / (int)sizeof(DT);
  Quad q;
  if (!quad_of(a, q)) return;
  const uint32_t scales = quad_scales(a, q)[threadIdx.x % kWave];
  const int width = (min(4 * kTileCols, a.K - q.k0) + PER - 1) / PER;  // lanes that a row takes
  if (width > kWave / 2) dequant_quad<1, WHOLE, DT>(a, q, scales, width);
  else if (width > kWave / 4) dequant_quad<2, WHOLE, DT>(a, q, scales, width);
  else dequant_quad<4, WHOLE, DT>(a, q, scales, width);
}

template <typename K>
hipError_t launch(K kern, const Fp4WeightsArgs &a, hipStream_t st) {
  const size_t quads = (size_t)a.mats * a.NT * a.KQ;
  return launch_kernel(kern, dim3((unsigned)((quads + kWaves - 1) / kWaves)), dim3(kThreads), 0, st, a);
}

// The one of two kernels that the rows take (both, where a first call loads them).
template <typename DT, typename K>
hipError_t launch_rows(K whole, K other, const Fp4WeightsArgs &a, hipStream_t st) {
  if (tl_resolve_only) {
    const hipError_t e = launch(whole, a, st);
    if (e != hipSuccess) return e;
  }
  return launch(whole_lines<DT>(a.K) && !tl_resolve_only ? whole : other, a, st);
}
template <typename DT> hipError_t quantize(const Fp4WeightsArgs &a, hipStream_t st) {
  return launch_rows<DT>(k_quant_fp4<true, DT>, k_quant_fp4<false, DT>, a, st);
}
template <typename DT> hipError_t dequantize(const Fp4WeightsArgs &a, hipStream_t st) {
  return launch_rows<DT>(k_dequant_fp4<true, DT>, k_dequant_fp4<false, DT>, a, st);
}

}  // namespace

hipError_t launch_quantize_fp4(const Fp4WeightsArgs &a, bool bf16, hipStream_t st) {
  return bf16 ? quantize<uint16_t>(a, st) : quantize<float>(a, st);
}

hipError_t launch_pack_fp4(const Fp4WeightsArgs &a, hipStream_t st) { return launch(k_pack_fp4, a, st); }

hipError_t launch_dequantize_fp4(const Fp4WeightsArgs &a, bool bf16, hipStream_t st) {
  return bf16 ? dequantize<uint16_t>(a, st) : dequantize<float>(a, st);
}

}  // namespace moelora
