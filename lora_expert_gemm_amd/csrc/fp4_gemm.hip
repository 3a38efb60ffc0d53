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

// --------------------------------------------------------------- many rows
//
// 16 TT token rows x 64 WT weight rows (SILU: half gate, half up) a workgroup
// of 4 waves; a wave owns WT weight tiles against all the tokens.  Slabs of 128
// columns: the tokens into LDS, where the waves share them, the weights into
// registers of the wave that uses them, one tile a load, a slab ahead.
//
// DMA: bf16 rows of whole 16-byte chunks go straight into two LDS stages, one
// slab ahead, with one barrier a slab; rows past the expert's last and chunks past
// K lie past the buffer resource's end, so their loads fetch nothing and give
// zeros.  Otherwise (float32 rows, in their three parts; bf16 rows of odd length) they pass
// through registers into one stage, between two barriers.
constexpr int kGWaves = 4, kGThreads = kGWaves * kWave;

// LDS byte offset of 16-byte chunk q of a 256-byte row: 16 consecutive rows read
// at one chunk fall on 16 distinct bank groups.
__device__ __forceinline__ int slab_off(int row, int q) { return row * 256 + ((q ^ (row & 15)) << 4); }

// 16 bytes a lane from `base` + voff + soff into 1 KB of LDS; zeros where they lie
// past `bytes`.
__device__ __forceinline__ void dma16(const void *base, int bytes, unsigned char *lds, uint32_t voff, int soff) {
  const __amdgpu_buffer_rsrc_t res =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, bytes, kBufferWord3);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(res, (__attribute__((address_space(3))) void *)lds, 16, voff, soff, 0, 0);
}

template <int WT, int TT, bool ONCE, bool DMA, bool SILU, typename DT>
__global__ __launch_bounds__(kGThreads, 2) void k_fp4_tiled(Fp4GemmArgs a, int ncols) {
  extern __shared__ __align__(16) unsigned char smem[];
  typedef Parts<DT> P;
  constexpr int HV = SILU ? 2 : 1, WH = WT / HV;  // weight tiles of a half
  constexpr int GM = 16 * TT, PLANE = GM * 256, STAGE = PLANE * P::kParts;
  static_assert(!DMA || sizeof(DT) == 2, "");
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int l16 = lane & 15, g = lane >> 4;
  const RowTile rt = find_tile(a, GM, ncols, blockIdx.x);
  if (rt.e < 0) return;
  const int rows = min(GM, rt.hi - rt.m0), KB = a.KB, K = a.K;
  const int t0 = (rt.nt * kGWaves + wave) * WH;  // the wave's first weight tile, in each half
  const uint8_t *wp[WT], *sp[WT];
#pragma unroll
  for (int i = 0; i < WT; ++i) {
    // (tiles past the last repeat it and are dropped)
    const size_t tile = ((size_t)rt.e * HV + i / WH) * a.NT + min(t0 + i % WH, a.NT - 1);
    wp[i] = a.w + tile * KB * kTileBytes;
    sp[i] = a.ws + tile * a.KQ * kScaleBytes;
  }
  struct Weights {
    u32x4_t c[WT];
    uint32_t s[WT];
  };
  auto load_w = [&](Weights &w, int b) {
    b = min(b, KB - 1);
#pragma unroll
    for (int i = 0; i < WT; ++i) {
      const u32x4_t *p = reinterpret_cast<const u32x4_t *>(wp[i] + (size_t)b * kTileBytes) + lane;
      w.c[i] = ONCE ? __builtin_nontemporal_load(p) : *p;
      w.s[i] = reinterpret_cast<const uint32_t *>(sp[i] + (size_t)(b / 4) * kScaleBytes)[lane];
    }
  };

  // ---- tokens
  constexpr int XD = GM / 4 / kGWaves;  // DMA loads a wave and slab, 4 rows each
  uint32_t xoff[DMA ? XD : 1], xtail[DMA ? XD : 1];
  if constexpr (DMA) {
#pragma unroll
    for (int j = 0; j < XD; ++j) {
      const int r = 4 * (XD * wave + j) + (lane >> 4), q = (lane & 15) ^ (r & 15);
      xoff[j] = (uint32_t)(r * K * 2 + q * 16);
      xtail[j] = (KB - 1) * kTileCols + 8 * q < K ? xoff[j] : 0x80000000u;
    }
  }
  const DT *const xrows = static_cast<const DT *>(a.x) + (size_t)rt.m0 * K;
  auto issue_x = [&](int b) {  // slab b by DMA into stage b % 2
    if constexpr (DMA) {
      unsigned char *st = smem + b % 2 * STAGE + XD * wave * 1024;
#pragma unroll
      for (int j = 0; j < XD; ++j)
        dma16(xrows, b < KB ? rows * K * 2 : 0, st + j * 1024, b == KB - 1 ? xtail[j] : xoff[j], b * 256);
    }
  };
  // through registers: chunk u of a thread is eight elements, 16 chunks a row
  constexpr int XR = GM * 16 / kGThreads;
  u32x4_t xr[DMA ? 1 : XR][P::kLoads];
  auto load_x = [&](int b) {
    if constexpr (!DMA) {
#pragma unroll
      for (int u = 0; u < XR; ++u) {
        const int c = u * kGThreads + tid, r = min(c / 16, rows - 1);  // (rows past the last are dropped)
        load8<DT>(xrows + (size_t)r * K, min(b, KB - 1) * kTileCols + c % 16 * 8, K, xr[u]);
      }
    }
  };
  auto store_x = [&]() {
    if constexpr (!DMA) {
#pragma unroll
      for (int u = 0; u < XR; ++u) {
        const int c = u * kGThreads + tid;
        const P p = P::of(xr[u]);
#pragma unroll
        for (int q = 0; q < P::kParts; ++q)
          *reinterpret_cast<u32x4_t *>(smem + q * PLANE + slab_off(c / 16, c % 16)) = p.p[q];
      }
    }
  };

  f32x4_t acc[WT][TT];
#pragma unroll
  for (int i = 0; i < WT; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[i][t] = f32x4_t{0, 0, 0, 0};

  // Slab b with its weights in `w`, and what is loaded meanwhile: the weights
  // of slab b + 1 into `wn`, its tokens.
  auto step = [&](int b, const Weights &w, Weights &wn) {
    if constexpr (DMA) {
      // this wave's tokens of b landed (the weights behind them may not have),
      // its reads of slab b - 1 done, for every wave
      __builtin_amdgcn_s_waitcnt(wait_vmcnt(2 * WT) & ~0x0f00);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      issue_x(b + 1);
      __builtin_amdgcn_sched_barrier(0);
      load_w(wn, b + 1);
      __builtin_amdgcn_sched_barrier(0);
    } else {
      __syncthreads();  // slab b - 1 is read out
      store_x();
      __syncthreads();
      load_w(wn, b + 1);
      load_x(b + 1);
    }
    const unsigned char *st = smem + (DMA ? b % 2 * STAGE : 0);
    float s[WT];
#pragma unroll
    for (int i = 0; i < WT; ++i) s[i] = scale_of_code(w.s[i] >> 8 * (b % 4) & 255u);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      u32x4_t wv[WT];
#pragma unroll
      for (int i = 0; i < WT; ++i) wv[i] = e2m1x8_to_bf16(w.c[i][c], s[i]);
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int q = 0; q < P::kParts; ++q) {
          const u32x4_t x = *reinterpret_cast<const u32x4_t *>(st + q * PLANE + slab_off(16 * t + l16, 4 * g + c));
#pragma unroll
          for (int i = 0; i < WT; ++i) Mma<uint16_t>::step(acc[i][t], wv[i], x);
        }
    }
  };

  Weights wa, wb;
  issue_x(0);
  __builtin_amdgcn_sched_barrier(0);
  load_w(wa, 0);
  load_x(0);
  int b = 0;
  for (; b + 1 < KB; b += 2) {
    step(b, wa, wb);
    step(b + 1, wb, wa);
  }
  if (b < KB) step(b, wa, wb);
  __builtin_amdgcn_s_waitcnt(0x0f70);  // no load of this workgroup outlives it

#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int m = 16 * t + l16;
    if (m >= rows) continue;
    DT *row = static_cast<DT *>(a.out) + (size_t)(rt.m0 + m) * a.N;
#pragma unroll
    for (int i = 0; i < WH; ++i) {
      const int n = (t0 + i) * kTileRows + 4 * g;
      if (n >= a.N) continue;
      float o[4];
#pragma unroll
      for (int v = 0; v < 4; ++v)
        o[v] = SILU ? silu_mul<sizeof(DT) == 4>(acc[i][t][v], acc[(i + WH) % WT][t][v]) : acc[i][t][v];
      store4<DT>(row, n, a.N, o);
    }
  }
}

template <int WT, int TT, bool ONCE, bool DMA, bool SILU, typename DT>
hipError_t tiled_t(const Fp4GemmArgs &a, hipStream_t st) {
  constexpr int TILES = kGWaves * WT / (SILU ? 2 : 1), GM = 16 * TT;
  constexpr int LDS = (DMA ? 2 : 1) * GM * 256 * Parts<DT>::kParts;
  auto kern = k_fp4_tiled<WT, TT, ONCE, DMA, SILU, DT>;
  hipError_t err = hipFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
  if (err != hipSuccess) return err;
  const int ncols = (a.NT + TILES - 1) / TILES;
  const int ne = a.E < a.R ? a.E : a.R;
  const int tiles = (int)(((long long)a.R + (long long)ne * (GM - 1)) / GM);
  return launch_kernel(kern, dim3(round_up8(tiles * ncols)), dim3(kGThreads), LDS, st, a, ncols);
}

template <int NT, int TG, bool SILU, typename DT>
hipError_t stream_t(const Fp4GemmArgs &a, hipStream_t st, int groups) {
  return launch_kernel(k_fp4_stream<NT, TG, SILU, DT>, dim3((a.NT + NT - 1) / NT, a.E < a.R ? a.E : a.R, groups),
                       dim3(kSThreads), 0, st, a);
}

// Most workgroups a tiled launch can hold: row tiles of GM rows (each expert's
// last one short) times column tiles.
long long tiled_wgs(const Fp4GemmArgs &a, bool silu, int WT, int TT) {
  const long long GM = 16 * TT, tiles = kGWaves * WT / (silu ? 2 : 1);
  const long long ne = a.E < a.R ? a.E : a.R;
  return (a.R + ne * (GM - 1)) / GM * ((a.NT + tiles - 1) / tiles);
}

Fp4Choice choose(const Fp4GemmArgs &a, bool silu, bool bf16) {
  const int mean = a.R / (a.E < a.R ? a.E : a.R);  // rows an expert, if all are hit
  if (mean <= 16) return {Fp4Kernel::kStream1, 1};
  if (bf16 && a.K % 8 == 0) {
    if (mean >= 96 && tiled_wgs(a, silu, 4, 8) >= 512) return {Fp4Kernel::kTile4x8, 1};
    if (mean > 40) return {Fp4Kernel::kTile4x4, 1};
    return {Fp4Kernel::kTile2x2Once, 1};
  }
  if (mean > 40) return {Fp4Kernel::kRegs4x4, 1};
  return {Fp4Kernel::kRegs2x2, 1};
}

template <bool SILU, typename DT>
hipError_t launch_t(const Fp4GemmArgs &a, Fp4Choice c, hipStream_t st) {
  constexpr int NT = SILU ? 1 : 2;
  switch (c.kernel) {
    case Fp4Kernel::kStream1: return stream_t<NT, 1, SILU, DT>(a, st, c.groups);
    case Fp4Kernel::kStream2: return stream_t<NT, 2, SILU, DT>(a, st, c.groups);
    case Fp4Kernel::kTile2x2Once:
      if constexpr (sizeof(DT) == 2) return tiled_t<2, 2, true, true, SILU, DT>(a, st);
      break;
    case Fp4Kernel::kTile2x4:
      if constexpr (sizeof(DT) == 2) return tiled_t<2, 4, false, true, SILU, DT>(a, st);
      break;
    case Fp4Kernel::kTile4x4:
      if constexpr (sizeof(DT) == 2) return tiled_t<4, 4, false, true, SILU, DT>(a, st);
      break;
    case Fp4Kernel::kTile4x8:
      if constexpr (sizeof(DT) == 2) return tiled_t<4, 8, false, true, SILU, DT>(a, st);
      break;
    case Fp4Kernel::kRegs2x2: return tiled_t<2, 2, false, false, SILU, DT>(a, st);
    case Fp4Kernel::kRegs4x4: return tiled_t<4, 4, false, false, SILU, DT>(a, st);
  }
  return hipErrorInvalidValue;
}

hipError_t launch(const Fp4GemmArgs &a, bool silu, bool bf16, Fp4Choice c, hipStream_t st) {
  if (silu) return bf16 ? launch_t<true, uint16_t>(a, c, st) : launch_t<true, float>(a, c, st);
  return bf16 ? launch_t<false, uint16_t>(a, c, st) : launch_t<false, float>(a, c, st);
}

}  // namespace

Fp4Choice choose_fp4_gemm(const Fp4GemmArgs &a, bool silu, bool bf16) { return choose(a, silu, bf16); }

hipError_t launch_fp4_gemm(const Fp4GemmArgs &a, bool silu, bool bf16, hipStream_t st) {
  return launch(a, silu, bf16, choose(a, silu, bf16), st);
}

hipError_t resolve_fp4_gemm(bool silu, bool bf16) {
  Fp4GemmArgs a{};
  a.R = a.N = a.K = a.E = a.NT = a.KB = a.KQ = 1;
  for (int k = 0; k < kFp4Kernels; ++k) {
    const Fp4Kernel kernel = (Fp4Kernel)k;
    if (!bf16 && fp4_needs_bf16(kernel)) continue;
    const hipError_t e = launch(a, silu, bf16, {kernel, 1}, nullptr);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moelora
