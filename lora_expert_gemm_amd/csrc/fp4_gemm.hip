// Grouped product of rows and 4-bit weights (E2M1 codes, one power of two a
// group of 32 along the contraction; layout in fp4.h):
//
//   out[m][n] = sum_k x[m][k] w[e][n][k]
//
// for the rows m of expert e, start[e] <= m < start[e + 1]; with SILU the
// weights are two matrices (gate, up) and out = SiLU(gate) * up.
//
// One conversion instruction turns two codes into two bf16 values with the
// group's scale in them, exactly, so the bf16 matrix core takes them as they are
// and no scaling is left for the sums: eight codes, one dword, are a lane's share
// of one v_mfma_f32_16x16x32_bf16 (weights on the row side, tokens on the
// column side).  A lane holds 32 neighbouring columns of its weight row, the
// i-th instruction takes the eight from 8 i on, and the tokens' operand is read
// to match.  float32 rows are cut into three bf16 parts (the upper, middle and
// lower eight bits of the significand: their sum is the value itself), and
// every part meets the weights in turn; sums are float32 throughout.
#include "common.h"
#include "fp4.h"
#include "grouped.h"
#include "kernels.h"
#include "ops.h"

namespace moelora {

namespace {

// Eight values of a row as MFMA operands whose sum they are.
template <typename DT> struct Parts;
template <> struct Parts<uint16_t> {
  static constexpr int kLoads = 1, kParts = 1;  // 16-byte loads for eight values
  u32x4_t p[1];
  __device__ __forceinline__ static Parts of(const u32x4_t *v) { return {{v[0]}}; }
};
template <> struct Parts<float> {
  static constexpr int kLoads = 2, kParts = 3;
  u32x4_t p[3];
  __device__ __forceinline__ static Parts of(const u32x4_t *v) {
    Parts r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[2], m[2], l[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t u = v[i / 2][i % 2 * 2 + j];
        const float f = __uint_as_float(u);
        const float f1 = f - __uint_as_float(u & 0xffff0000u);  // exact
        const float f2 = f1 - __uint_as_float(__float_as_uint(f1) & 0xffff0000u);
        h[j] = u, m[j] = __float_as_uint(f1), l[j] = __float_as_uint(f2);
      }
      // the upper halves side by side
      r.p[0][i] = __builtin_amdgcn_perm(h[1], h[0], 0x07060302u);
      r.p[1][i] = __builtin_amdgcn_perm(m[1], m[0], 0x07060302u);
      r.p[2][i] = __builtin_amdgcn_perm(l[1], l[0], 0x07060302u);
    }
    return r;
  }
};

// Elements c .. c + 7 of a row of K as they are stored, zeros past K.  Whole
// ones are 16-byte loads, which need no more than 2-byte alignment here.
template <typename DT>
__device__ __forceinline__ void load8(const DT *row, int c, int K, u32x4_t *v) {
  typedef u32x4_t mem __attribute__((aligned(2)));
  constexpr int n = Parts<DT>::kLoads, per = 16 / sizeof(DT);
  if (c + 8 <= K) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = *reinterpret_cast<const mem *>(row + c + per * i);
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      Chunk<DT> e;
#pragma unroll
      for (int j = 0; j < per; ++j) e.v[j] = c + per * i + j < K ? row[c + per * i + j] : DT(0);
      v[i] = __builtin_bit_cast(u32x4_t, e);
    }
  }
}

// ---------------------------------------------------------------- few rows
//
// A workgroup owns NT tiles of 16 weight rows (of each half) of one expert and
// up to 16 TG of its tokens at a time (every gridDim.z-th group); its four waves take every
// fourth tile along the contraction and add their sums through LDS in wave
// order, so that a narrow product still fills the chip.  Weights go from memory
// straight into registers, 1 KB a load.
constexpr int kSWaves = 4;
constexpr int kSThreads = kSWaves * kWave;

template <int NT, int TG, bool SILU, typename DT>
__global__ __launch_bounds__(kSThreads) void k_fp4_stream(Fp4GemmArgs a) {
  constexpr int HV = SILU ? 2 : 1, A = HV * NT, XL = Parts<DT>::kLoads;
  __shared__ f32x4_t red[kSWaves][A * TG][kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int l16 = lane & 15, g = lane >> 4;
  int e, lo, hi;
  if (!find_expert(a, blockIdx.y, e, lo, hi)) return;
  const int KB = a.KB, t0 = blockIdx.x * NT;
  const uint8_t *wp[A], *sp[A];
#pragma unroll
  for (int i = 0; i < A; ++i) {
    // (tiles past the last repeat it and are dropped)
    const size_t tile = ((size_t)e * HV + i / NT) * a.NT + min(t0 + i % NT, a.NT - 1);
    wp[i] = a.w + tile * KB * kTileBytes + lane * 16;
    sp[i] = a.ws + tile * a.KQ * kScaleBytes + lane * 4;
  }
  for (int m0 = lo + blockIdx.z * 16 * TG; m0 < hi; m0 += gridDim.z * 16 * TG) {
    f32x4_t acc[A][TG];
#pragma unroll
    for (int i = 0; i < A; ++i)
#pragma unroll
      for (int t = 0; t < TG; ++t) acc[i][t] = f32x4_t{0, 0, 0, 0};
    const DT *xp[TG];
#pragma unroll
    for (int t = 0; t < TG; ++t)  // (rows past the last repeat it and are dropped)
      xp[t] = static_cast<const DT *>(a.x) + (size_t)min(m0 + 16 * t + l16, hi - 1) * a.K;
    for (int b = wave; b < KB; b += kSWaves) {
      u32x4_t w[A];
      float s[A];
#pragma unroll
      for (int i = 0; i < A; ++i) {
        w[i] = *reinterpret_cast<const u32x4_t *>(wp[i] + (size_t)b * kTileBytes);
        const uint32_t four = *reinterpret_cast<const uint32_t *>(sp[i] + (size_t)(b / 4) * kScaleBytes);
        s[i] = scale_of_code(four >> 8 * (b % 4) & 255u);
      }
#pragma unroll
      for (int t = 0; t < TG; ++t) {
        u32x4_t v[4][XL];
#pragma unroll
        for (int c = 0; c < 4; ++c) load8<DT>(xp[t], b * kTileCols + g * kGroup + 8 * c, a.K, v[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const Parts<DT> x = Parts<DT>::of(v[c]);
#pragma unroll
          for (int i = 0; i < A; ++i) {
            const u32x4_t wv = e2m1x8_to_bf16(w[i][c], s[i]);
#pragma unroll
            for (int p = 0; p < Parts<DT>::kParts; ++p) Mma<uint16_t>::step(acc[i][t], wv, x.p[p]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < A; ++i)
#pragma unroll
      for (int t = 0; t < TG; ++t) red[wave][i * TG + t][lane] = acc[i][t];
    __syncthreads();
    // one wave per (tile, token group): the four waves' sums in wave order
    for (int q = wave; q < NT * TG; q += kSWaves) {
      const int i = q / TG, t = q % TG;
      f32x4_t v[HV];
#pragma unroll
      for (int h = 0; h < HV; ++h) {
        const int at = (h * NT + i) * TG + t;
        v[h] = red[0][at][lane];
#pragma unroll
        for (int w = 1; w < kSWaves; ++w) {
          const f32x4_t o = red[w][at][lane];
#pragma unroll
          for (int c = 0; c < 4; ++c) v[h][c] += o[c];
        }
      }
      const int m = m0 + 16 * t + l16, n = (t0 + i) * kTileRows + 4 * g;
      if (m < hi && n < a.N) {
        float o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = SILU ? silu_mul<sizeof(DT) == 4>(v[0][c], v[HV - 1][c]) : v[0][c];
        store4<DT>(static_cast<DT *>(a.out) + (size_t)m * a.N, n, a.N, o);
      }
    }
    __syncthreads();
  }
}

template <bool SILU, typename DT>
hipError_t stream_t(const Fp4GemmArgs &a, hipStream_t st) {
  constexpr int NT = SILU ? 1 : 2;
  const int ne = a.E < a.R ? a.E : a.R, mean = a.R / ne;
  const int rows = mean <= 16 ? 16 : 32, groups = (mean + rows - 1) / rows;
  const dim3 grid((a.NT + NT - 1) / NT, ne, groups < 1024 ? groups : 1024);
  if (rows == 16 || tl_resolve_only) {
    const hipError_t e = launch_kernel(k_fp4_stream<NT, 1, SILU, DT>, grid, dim3(kSThreads), 0, st, a);
    if (!tl_resolve_only || e != hipSuccess) return e;
  }
  return launch_kernel(k_fp4_stream<NT, 2, SILU, DT>, grid, dim3(kSThreads), 0, st, a);
}

}  // namespace

hipError_t launch_fp4_gemm(const Fp4GemmArgs &a, bool silu, bool bf16, hipStream_t st) {
  if (silu) return bf16 ? stream_t<true, uint16_t>(a, st) : stream_t<true, float>(a, st);
  return bf16 ? stream_t<false, uint16_t>(a, st) : stream_t<false, float>(a, st);
}

}  // namespace moelora
