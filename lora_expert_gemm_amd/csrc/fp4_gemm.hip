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
// lower eight bits of the significand: their sum is the value itself from 2^-110 on,
// below that the value cut to a multiple of 2^-133, bf16's smallest step), and
// every part meets the weights in turn; sums are float32 throughout.
#include <algorithm>

#include "common.h"
#include "fp4.h"
#include "grouped.h"
#include "kernels.h"
#include "ops.h"

namespace moelora {

namespace {

// Eight values of a row as MFMA operands whose sum they are.  INF: of infinities too,
// which are their own upper part; without it inf - inf makes the lower ones NaN.  Every
// contraction is made without it first (with it 2 to 3 % slower, one row 12 %), and where
// a sum then is NaN once more with it.
template <typename DT> struct Parts;
template <> struct Parts<uint16_t> {
  static constexpr int kLoads = 1, kParts = 1;  // 16-byte loads for eight values
  u32x4_t p[1];
  template <bool INF> __device__ __forceinline__ static Parts of(const u32x4_t *v) { return {{v[0]}}; }
};
template <> struct Parts<float> {
  static constexpr int kLoads = 2, kParts = 3;
  u32x4_t p[3];
  template <bool INF> __device__ __forceinline__ static Parts of(const u32x4_t *v) {
    Parts r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[2], m[2], l[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t u = v[i / 2][i % 2 * 2 + j];
        const float f = __uint_as_float(u);
        float f1 = f - __uint_as_float(u & 0xffff0000u);  // exact
        if (INF && __builtin_isinf(f)) f1 = 0.f;
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

// Whether one of a lane's sums is NaN (or two are infinities of either sign).
template <int N, int M> __device__ __forceinline__ bool some_nan(const f32x4_t (&acc)[N][M]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < M; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) s += acc[i][j][c];
  return s != s;
}

// v shifted right by 0 <= n <= 16 bytes.
__device__ __forceinline__ u32x4_t shift_right(u32x4_t v, int n) {
  typedef unsigned long long u64;
  u64 lo = (u64)v[1] << 32 | v[0], hi = (u64)v[3] << 32 | v[2];
  const int bits = 8 * n & 63;
  if (n >= 8) lo = hi, hi = 0;
  if (n >= 16) lo = 0;
  lo = lo >> bits | (hi << 1) << (63 - bits);
  hi >>= bits;
  return u32x4_t{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// Elements c .. c + 7 of the row of K (16 bytes or more) that starts `row` elements behind `base`, as
// 16-byte loads, which need no more than 2-byte alignment here.  One that would
// pass the row's end is moved back to end with it; fix8 shifts it to its place,
// zeros behind, where the values are needed, so that the load itself need not be
// waited for.
template <typename DT> constexpr int kPerLoad = 16 / (int)sizeof(DT);
template <typename DT>
__device__ __forceinline__ void load8(const DT *base, uint32_t row, int c, int K, u32x4_t *v) {
  typedef u32x4_t mem __attribute__((aligned(2)));
  constexpr int per = kPerLoad<DT>;
#pragma unroll
  for (int i = 0; i < Parts<DT>::kLoads; ++i) {
    const int k = c + per * i;
    const uint32_t at = (row + min(k, K - per)) * (uint32_t)sizeof(DT);
    v[i] = *reinterpret_cast<const mem *>(reinterpret_cast<const char *>(base) + at);
  }
}
template <typename DT> __device__ __forceinline__ void fix8(int c, int K, u32x4_t *v) {
  constexpr int per = kPerLoad<DT>;
#pragma unroll
  for (int i = 0; i < Parts<DT>::kLoads; ++i)
    v[i] = shift_right(v[i], max(0, min(c + per * i - (K - per), per)) * (int)sizeof(DT));
}

// A wave's weights: WH neighbouring rows of tiles in each of HV matrices.
template <int HV, int WH> struct TileRows {
  const uint8_t *codes[HV], *scales[HV];
  uint32_t at[WH], sat[WH];  // a lane's place in each row of tiles
  int bytes, sbytes;         // of the rows that exist

  __device__ __forceinline__ TileRows(const Fp4GemmArgs &a, int e, int t0, int lane) {
    const int n = max(0, min(WH, a.NT - t0));
    bytes = n * a.KB * kTileBytes, sbytes = n * a.KQ * kScaleBytes;
#pragma unroll
    for (int h = 0; h < HV; ++h) {
      const size_t row = ((size_t)e * HV + h) * a.NT + (n ? t0 : 0);
      codes[h] = a.w + row * a.KB * kTileBytes, scales[h] = a.ws + row * a.KQ * kScaleBytes;
    }
#pragma unroll
    for (int i = 0; i < WH; ++i) {
      at[i] = i * a.KB * kTileBytes + lane * 16, sat[i] = i * a.KQ * kScaleBytes + lane * 4;
    }
  }
};
// A wave's tiles of slab b: a lane's 32 codes, and the scales of its groups in
// slabs b / 4 * 4 .. + 3.  Rows that do not exist, and slabs past the last, lie
// past their buffer resource's end: they fetch nothing and give zeros.
template <int A> struct Weights {
  u32x4_t c[A];
  uint32_t s[A];
};
template <bool ONCE, int HV, int WH>
__device__ __forceinline__ void load_weights(Weights<HV * WH> &w, const TileRows<HV, WH> &r, int KB, int b) {
#pragma unroll
  for (int h = 0; h < HV; ++h) {
    const __amdgpu_buffer_rsrc_t codes = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(r.codes[h]), (short)0, b < KB ? r.bytes : 0, kBufferWord3);
    const __amdgpu_buffer_rsrc_t scales = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(r.scales[h]), (short)0, b < KB ? r.sbytes : 0, kBufferWord3);
#pragma unroll
    for (int i = 0; i < WH; ++i) {
      w.c[h * WH + i] =
          __builtin_amdgcn_raw_buffer_load_b128(codes, r.at[i], b * kTileBytes, ONCE ? kCpolNonTemporal : 0);
      w.s[h * WH + i] = __builtin_amdgcn_raw_buffer_load_b32(scales, r.sat[i], b / 4 * kScaleBytes, 0);
    }
  }
}

// ---------------------------------------------------------------- few rows
//
// A workgroup owns NT tiles of 16 weight rows (of each half) of one expert and
// up to 16 of its tokens at a time (every gridDim.z-th group); its W waves take every
// W-th tile along the contraction, one ahead, and add their sums through LDS in
// wave order, so that a narrow product still fills the chip.  Weights go from
// memory straight into registers, 1 KB a load, tokens too.  Bound by the weights' bytes:
// 64 rows on 23 of 32 experts, 2880 -> 2 x 2880 38 us, 5.75 TB/s; one row, 4096 -> 11008, 7.6,
// one round of 344 workgroups whose start and end weigh as much as their loads.
template <int NT, int W, bool ONCE, bool SILU, typename DT>
__global__ __launch_bounds__(W * kWave) void k_fp4_stream(Fp4GemmArgs a) {
  constexpr int HV = SILU ? 2 : 1, A = HV * NT, XL = Parts<DT>::kLoads;
  __shared__ f32x4_t red[W][A][kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int l16 = lane & 15, g = lane >> 4;
  int e, lo, hi;
  if (!find_expert(a, blockIdx.y, e, lo, hi)) return;
  e = __builtin_amdgcn_readfirstlane(e);
  const int KB = a.KB, K = a.K, t0 = blockIdx.x * NT;
  const TileRows<HV, NT> tr(a, e, t0, lane);
  for (int m0 = lo + blockIdx.z * 16; m0 < hi; m0 += gridDim.z * 16) {
    f32x4_t acc[1][A];
    const DT *const xrows = static_cast<const DT *>(a.x) + (size_t)m0 * K;
    const uint32_t row = (uint32_t)min(l16, hi - m0 - 1) * K;  // (rows past the last repeat it and are dropped)
    struct Slab {
      Weights<A> w;
      u32x4_t x[4][XL];
    };
    auto load = [&](Slab &v, int b) {
      load_weights<ONCE, HV, NT>(v.w, tr, KB, b);
#pragma unroll
      for (int c = 0; c < 4; ++c) load8<DT>(xrows, row, b * kTileCols + g * kGroup + 8 * c, K, v.x[c]);
    };
    static_assert(W % 4 == 0, "a wave's slabs have one place in the scales' fours");
    const auto contract = [&]<bool INF>() {
#pragma unroll
      for (int i = 0; i < A; ++i) acc[0][i] = f32x4_t{0, 0, 0, 0};
      Slab v;
      load(v, wave);
      for (int b = wave; b < KB; b += W) {
        if ((b + 1) * kTileCols > K) {
#pragma unroll
          for (int c = 0; c < 4; ++c) fix8<DT>(b * kTileCols + g * kGroup + 8 * c, K, v.x[c]);
        }
        float s[A];
#pragma unroll
        for (int i = 0; i < A; ++i) s[i] = scale_of_code(v.w.s[i] >> 8 * (wave % 4) & 255u);  // (b % 4 is wave % 4)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          u32x4_t wv[A];
#pragma unroll
          for (int i = 0; i < A; ++i) wv[i] = e2m1x8_to_bf16(v.w.c[i][c], s[i]);
          const Parts<DT> x = Parts<DT>::template of<INF>(v.x[c]);
#pragma unroll
          for (int q = 0; q < Parts<DT>::kParts; ++q)
#pragma unroll
            for (int i = 0; i < A; ++i) Mma<uint16_t>::step(acc[0][i], wv[i], x.p[q]);
        }
        load(v, b + W);
      }
    };
    contract.template operator()<false>();
    if constexpr (Parts<DT>::kParts > 1) {
      if (__builtin_expect(__any(some_nan(acc)), 0)) contract.template operator()<true>();
    }
#pragma unroll
    for (int i = 0; i < A; ++i) red[wave][i][lane] = acc[0][i];
    __syncthreads();
    // one wave per tile: the waves' sums in wave order
    for (int i = wave; i < NT; i += W) {
      f32x4_t v[HV];
#pragma unroll
      for (int h = 0; h < HV; ++h) {
        v[h] = red[0][h * NT + i][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) {
          const f32x4_t o = red[w][h * NT + i][lane];
#pragma unroll
          for (int c = 0; c < 4; ++c) v[h][c] += o[c];
        }
      }
      const int m = m0 + l16, n = (t0 + i) * kTileRows + 4 * g;
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
// 16 TT token rows x 64 WT weight rows (SILU: half gate, half up) a workgroup;
// KS groups of 4 waves take every KS-th slab of 128 columns each and add their
// sums through LDS in the end, in their order.  A wave owns WT weight tiles against all the
// tokens.  Per slab and group: the tokens into one of two LDS stages, where the waves
// share them, the weights, a slab ahead, into registers of the wave that uses them, one tile a
// load; one barrier.
//
// DMA: bf16 rows of whole 16-byte chunks go straight into LDS, a slab ahead;
// rows past the expert's last and chunks past K lie past the buffer resource's
// end, so their loads fetch nothing and give zeros.  Otherwise (float32 rows, in
// their three parts; bf16 rows of any length) they pass through registers, a slab
// ahead of their stage.
//
// Many rows are bound by the matrix cores: 25600 rows of 32 experts, 2880 -> 2 x 2880 with
// SILU 680 us, 1.25 PFLOP/s (8192^3 1.39, as the library's bf16 product), the cores busy 70 %
// of the cycles.  With some 20 rows an expert (2664 float32 rows of 128, 2050 -> 771, 48 us) a
// slab's latency and the weights' conversion weigh as much as the products: cores busy 32 %.
constexpr int kGWaves = 4, kGThreads = kGWaves * kWave;

// LDS byte offset of 16-byte chunk q of a 256-byte row: 16 consecutive rows read
// at one chunk fall on 16 distinct bank groups.  (Lanes of two chunks are served together
// and may meet, 3.8 cycles a read; an order in which none do was no faster.)
__device__ __forceinline__ int slab_off(int row, int q) { return row * 256 + ((q ^ (row & 15)) << 4); }

// Results of a token, WH neighbouring weight tiles from column n0 on, lane g holding
// columns 4 g .. + 3 of each: two tiles' lanes g and g + 1 change places, so that a lane
// has eight columns of one tile and stores 16 bytes, 64 of a row side by side (8 and 32
// without: 10750 rows of 23 experts 71 -> 1268 14.9 -> 14.0 us, 4096 of 32 gate_up 144 -> 140).
template <int WH>
__device__ __forceinline__ void store_pairs(uint16_t *row, bool some, int n0, int g, int N, const float (*o)[4]) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  typedef u32x4_t mem __attribute__((aligned(2)));
#pragma unroll
  for (int i = 0; i < WH; i += 2) {
    uint32_t a[2], b[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      a[v] = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)o[i][2 * v], (__bf16)o[i][2 * v + 1]});
      b[v] = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)o[i + 1][2 * v], (__bf16)o[i + 1][2 * v + 1]});
      // rows of 16 lanes: a's odd ones change places with b's even ones
      const auto s = __builtin_amdgcn_permlane16_swap(a[v], b[v], false, false);
      a[v] = s[0], b[v] = s[1];
    }
    const int n = n0 + (i + (g & 1)) * kTileRows + 8 * (g >> 1);
    const u32x4_t w = {a[0], a[1], b[0], b[1]};
    if (!some) continue;
    if (n + 8 <= N) {
      *reinterpret_cast<mem *>(row + n) = w;
    } else {
      const Chunk<uint16_t> e = chunk_elems<uint16_t>(w);
#pragma unroll
      for (int v = 0; v < 8; ++v)
        if (n + v < N) row[n + v] = e.v[v];
    }
  }
}

// 16 bytes a lane from `base` + voff + soff into 1 KB of LDS; zeros where they lie
// past `bytes`.
__device__ __forceinline__ void dma16(const void *base, int bytes, unsigned char *lds, uint32_t voff, int soff) {
  const __amdgpu_buffer_rsrc_t res =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, bytes, kBufferWord3);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(res, (__attribute__((address_space(3))) void *)lds, 16, voff, soff, 0, 0);
}

template <int WT, int TT, int KS, bool ONCE, bool DMA, bool SILU, typename DT>
__global__ __launch_bounds__(KS * kGThreads, KS > 1 || WT * TT <= 4 ? 4 : WT * TT <= 8 || DMA ? 3 : 2) void k_fp4_tiled(
    Fp4GemmArgs a, int ncols) {
  extern __shared__ __align__(16) unsigned char smem[];
  typedef Parts<DT> P;
  constexpr int HV = SILU ? 2 : 1, WH = WT / HV;  // weight tiles of a half
  constexpr int GM = 16 * TT, PLANE = GM * 256, STAGE = PLANE * P::kParts;
  static_assert(!DMA || sizeof(DT) == 2, "");
  const int tid = threadIdx.x % kGThreads, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int kg = __builtin_amdgcn_readfirstlane(threadIdx.x / kGThreads);
  const int l16 = lane & 15, g = lane >> 4;
  const RowTile rt = find_tile(a, GM, ncols, blockIdx.x);
  if (rt.e < 0) return;
  const int rows = min(GM, rt.hi - rt.m0), KB = a.KB, K = a.K;
  const int t0 = (rt.nt * kGWaves + wave) * WH;  // the wave's first weight tile, in each half
  const TileRows<HV, WH> tr(a, rt.e, t0, lane);
  const DT *const xrows = static_cast<const DT *>(a.x) + (size_t)rt.m0 * K;
  unsigned char *const stages = smem + kg * 2 * STAGE;

  // ---- tokens by DMA, 4 rows a load: slab b into stage s
  constexpr int XD = DMA ? GM / 4 / kGWaves : 1;
  uint32_t xoff[XD], xtail[XD];
#pragma unroll
  for (int j = 0; j < XD; ++j) {
    const int r = 4 * (XD * wave + j) + (lane >> 4), q = (lane & 15) ^ (r & 15);
    xoff[j] = (uint32_t)(r * K * 2 + q * 16);
    xtail[j] = (KB - 1) * kTileCols + 8 * q < K ? xoff[j] : 0x80000000u;
  }
  auto issue_x = [&](int b, int s) {
    unsigned char *st = stages + s * STAGE + XD * wave * 1024;
#pragma unroll
    for (int j = 0; j < XD; ++j)
      dma16(xrows, b < KB ? rows * K * 2 : 0, st + j * 1024, b == KB - 1 ? xtail[j] : xoff[j], b * 256);
  };
  // ---- or through registers: XR chunks of eight elements a thread, 16 a row
  constexpr int XR = DMA ? 1 : GM * 16 / kGThreads;
  struct Rows {
    u32x4_t v[XR][P::kLoads];
  };
  auto load_x = [&](Rows &x, int b) {
#pragma unroll
    for (int u = 0; u < XR; ++u) {
      const int c = u * kGThreads + tid, r = min(c / 16, rows - 1);  // (rows past the last are dropped)
      load8<DT>(xrows, (uint32_t)r * K, b * kTileCols + c % 16 * 8, K, x.v[u]);
    }
  };
  auto store_x = [&]<bool INF>(Rows &x, int b, int s) {
    unsigned char *st = stages + s * STAGE;
#pragma unroll
    for (int u = 0; u < XR; ++u) {
      const int c = u * kGThreads + tid;
      if ((b + 1) * kTileCols > K) fix8<DT>(b * kTileCols + c % 16 * 8, K, x.v[u]);
      const P p = P::template of<INF>(x.v[u]);
#pragma unroll
      for (int q = 0; q < P::kParts; ++q)
        *reinterpret_cast<u32x4_t *>(st + q * PLANE + slab_off(c / 16, c % 16)) = p.p[q];
    }
  };

  f32x4_t acc[WT][TT];
  // The group's i-th slab with its weights in `w`, and what is loaded meanwhile: the
  // next one's weights into `wn`, its rows (and those of the one after).
  Rows x;
  auto step = [&]<bool INF>(int i, const Weights<WT> &w, Weights<WT> &wn) {
    const int b = kg + i * KS, s = i & 1;
    if constexpr (DMA) {
      // this wave's tokens of b landed (the weights behind them may not have),
      // its reads of the slab before done, for every wave
      __builtin_amdgcn_s_waitcnt(wait_vmcnt(2 * WT) & ~0x0f00);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      issue_x(b + KS, s ^ 1);
      __builtin_amdgcn_sched_barrier(0);
      load_weights<ONCE, HV, WH>(wn, tr, KB, b + KS);
      __builtin_amdgcn_sched_barrier(0);
    } else {
      __syncthreads();  // slab b is stored, the one before read out
      store_x.template operator()<INF>(x, b + KS, s ^ 1);
      load_x(x, b + 2 * KS);
      load_weights<ONCE, HV, WH>(wn, tr, KB, b + KS);
    }
    if (t0 >= a.NT) return;  // (a wave without columns only helps with the tokens)
    const unsigned char *st = stages + s * STAGE;
    float sc[WT];
#pragma unroll
    for (int i = 0; i < WT; ++i) sc[i] = scale_of_code(w.s[i] >> 8 * (b % 4) & 255u);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      u32x4_t wv[WT];
#pragma unroll
      for (int i = 0; i < WT; ++i) wv[i] = e2m1x8_to_bf16(w.c[i][c], sc[i]);
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int q = 0; q < P::kParts; ++q) {
          const u32x4_t v = *reinterpret_cast<const u32x4_t *>(st + q * PLANE + slab_off(16 * t + l16, 4 * g + c));
#pragma unroll
          for (int i = 0; i < WT; ++i) Mma<uint16_t>::step(acc[i][t], wv[i], v);
        }
    }
  };

  const auto contract = [&]<bool INF>() {
#pragma unroll
    for (int i = 0; i < WT; ++i)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[i][t] = f32x4_t{0, 0, 0, 0};
    Weights<WT> wa, wb;
    if constexpr (DMA) {
      issue_x(kg, 0);
      __builtin_amdgcn_sched_barrier(0);
    } else {
      load_x(x, kg);
    }
    load_weights<ONCE, HV, WH>(wa, tr, KB, kg);
    if constexpr (!DMA) {
      store_x.template operator()<INF>(x, kg, 0);
      load_x(x, kg + KS);
    }
    // (every group makes as many steps, one barrier each; slabs past the last are zeros)
    const int steps = (KB + KS - 1) / KS;
    int i = 0;
    for (; i + 1 < steps; i += 2) {
      step.template operator()<INF>(i, wa, wb);
      step.template operator()<INF>(i + 1, wb, wa);
    }
    if (i < steps) step.template operator()<INF>(i, wa, wb);
    __builtin_amdgcn_s_waitcnt(0x0f70);  // no load of this workgroup outlives it
  };
  __shared__ int again;  // (cleared before the first step's barrier, set behind the last one's)
  if (P::kParts > 1 && threadIdx.x == 0) again = 0;
  contract.template operator()<false>();
  if (P::kParts > 1 && some_nan(acc)) again = 1;
  if constexpr (P::kParts > 1 || KS > 1) __syncthreads();  // no stage is written again while it is read
  if constexpr (P::kParts > 1) {
    if (__builtin_expect(__builtin_amdgcn_readfirstlane(again), 0)) {
      contract.template operator()<true>();
      __syncthreads();
    }
  }

  if constexpr (KS > 1) {
    f32x4_t *const sums = reinterpret_cast<f32x4_t *>(smem) + tid;
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < WT; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t) sums[((kg - 1) * WT * TT + i * TT + t) * kGThreads] = acc[i][t];
    }
    __syncthreads();
    if (kg > 0) return;
#pragma unroll
    for (int i = 0; i < WT; ++i)
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int q = 0; q < KS - 1; ++q) {
          const f32x4_t o = sums[(q * WT * TT + i * TT + t) * kGThreads];
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][t][v] += o[v];
        }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int m = 16 * t + l16;
    DT *row = static_cast<DT *>(a.out) + (size_t)(rt.m0 + min(m, rows - 1)) * a.N;
    float o[WH][4];
#pragma unroll
    for (int i = 0; i < WH; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        o[i][v] = SILU ? silu_mul<sizeof(DT) == 4>(acc[i][t][v], acc[(i + WH) % WT][t][v]) : acc[i][t][v];
    if constexpr (sizeof(DT) == 2 && WH % 2 == 0) {
      store_pairs<WH>(row, m < rows, t0 * kTileRows, g, a.N, o);
    } else {
#pragma unroll
      for (int i = 0; i < WH; ++i) {
        const int n = (t0 + i) * kTileRows + 4 * g;
        if (m < rows && n < a.N) store4<DT>(row, n, a.N, o[i]);
      }
    }
  }
}

// -------------------------------------------------------------- short rows
//
// Rows of less than 16 bytes: a thread a column, its few weights in registers,
// every gridDim.z-th row of the expert.
template <bool SILU, typename DT>
__global__ __launch_bounds__(256) void k_fp4_short(Fp4GemmArgs a) {
  constexpr int HV = SILU ? 2 : 1, MOST = 16 / (int)sizeof(DT) - 1;
  int e, lo, hi;
  if (!find_expert(a, blockIdx.y, e, lo, hi)) return;
  const int n = blockIdx.x * 256 + threadIdx.x, r = n % kTileRows;
  if (n >= a.N) return;
  float w[HV][MOST];
#pragma unroll
  for (int h = 0; h < HV; ++h) {
    const size_t tile = ((size_t)e * HV + h) * a.NT + n / kTileRows;
    const uint32_t c = *reinterpret_cast<const uint32_t *>(a.w + tile * kTileBytes + 16 * r);
    const float s = scale_of_code(a.ws[tile * kScaleBytes + 4 * r]);
    const u32x4_t v = e2m1x8_to_bf16(c, s);
#pragma unroll
    for (int k = 0; k < MOST; ++k) w[h][k] = __uint_as_float(k % 2 ? v[k / 2] & 0xffff0000u : v[k / 2] << 16);
  }
  for (int m = lo + blockIdx.z; m < hi; m += gridDim.z) {
    const DT *x = static_cast<const DT *>(a.x) + (size_t)m * a.K;
    float y[HV];
#pragma unroll
    for (int h = 0; h < HV; ++h) y[h] = 0.f;
#pragma unroll
    for (int k = 0; k < MOST; ++k) {
      if (k >= a.K) break;
#pragma unroll
      for (int h = 0; h < HV; ++h) y[h] = fmaf(Elem<DT>::to_f32(x[k]), w[h][k], y[h]);
    }
    static_cast<DT *>(a.out)[(size_t)m * a.N + n] =
        Elem<DT>::from_f32(SILU ? silu_mul<sizeof(DT) == 4>(y[0], y[HV - 1]) : y[0]);
  }
}

template <int WT, int TT, int KS, bool ONCE, bool DMA, bool SILU, typename DT>
hipError_t tiled_t(const Fp4GemmArgs &a, hipStream_t st) {
  constexpr int TILES = kGWaves * WT / (SILU ? 2 : 1), GM = 16 * TT;
  constexpr int SLABS = 2 * KS * GM * 256 * Parts<DT>::kParts, SUMS = (KS - 1) * kGThreads * WT * TT * 16;
  constexpr int LDS = SLABS > SUMS ? SLABS : SUMS;  // (the sums lie where the slabs were)
  static_assert(LDS <= 160 * 1024, "");
  auto kern = k_fp4_tiled<WT, TT, KS, ONCE, DMA, SILU, DT>;
  hipError_t err = hipFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
  if (err != hipSuccess) return err;
  const int ncols = (a.NT + TILES - 1) / TILES;
  const int ne = a.E < a.R ? a.E : a.R;
  const int tiles = (int)(((long long)a.R + (long long)ne * (GM - 1)) / GM);
  return launch_kernel(kern, dim3(round_up8(tiles * ncols)), dim3(KS * kGThreads), LDS, st, a, ncols);
}

template <int NT, int W, bool ONCE, bool SILU, typename DT>
hipError_t stream_t(const Fp4GemmArgs &a, hipStream_t st, int groups) {
  return launch_kernel(k_fp4_stream<NT, W, ONCE, SILU, DT>,
                       dim3((a.NT + NT - 1) / NT, a.E < a.R ? a.E : a.R, groups), dim3(W * kWave), 0, st, a);
}

// Most workgroups a launch of row groups of GM rows (each expert's last one short) and
// column groups of `tiles` weight tiles can hold.
long long workgroups(const Fp4GemmArgs &a, int GM, int tiles) {
  const long long ne = a.E < a.R ? a.E : a.R;
  return (a.R + ne * (GM - 1)) / GM * ((a.NT + tiles - 1) / tiles);
}

// Which kernel, by the mean rows of an expert and by how many workgroups it leaves
// (256 CUs); the host knows no more of the rows than their mean, so rows that crowd on few
// experts may take a slower one: 1024 rows, 2880 -> 2 x 2880 with SILU, bf16, are streamed for
// 256 experts, 348 us of even rows, 242 with all on two experts (41 by 4x4), where at most four
// workgroups a column group go through an expert's groups of 16 rows and its weights each time.
// us on one card; "g": by tokens, 32 experts, top-4, 2880 -> 2 x 2880 with
// SILU, bf16; "d": by rows, one expert, 4096 -> 11008.
//   few rows, many experts: four weight tiles a workgroup without LDS against tiles whose
//     tokens go through it: g16 37 / 43 (4x2), g64 57 / 48, g128 96 / 62 (16 tokens of
//     float32 58 / 51, by 4x1: they stay with tiles)
//   few rows, few workgroups: two weight tiles and eight waves on the contraction: d1 7.1
//     (four tiles and waves 8.6, split tiles 7.8)
//   little work: tiles with the contraction split over four groups of waves.  1x1: d16 8.0
//     (streamed 9.5 to 12, not split 17), 16 experts x 8 rows 4000 -> 500 8.0 (10.8), d64 16.2;
//     2x2: d64 13.0 (not split 20), 256 rows 4096 -> 4096 13.4 (17.4), 1000 rows of 8 experts
//     8000 -> 300 24 (29 by 1x1); float32 4x1: d64 23 (30).  Its sixteen
//     waves fill a CU: with more workgroups than CUs 2300 rows of 5 experts 1024 -> 446 12.6
//     (7.6 by 2x2 by DMA, which they take, 9.0 by 4x2), 3735 float32 rows of 94 948 -> 98 19.7
//     (14.3; with four column groups and more the rows come from caches, 1024 rows of 8
//     2048 -> 625 14.6 (17.1))
//   float32: 4x1 against 4x2, 21 rows an expert of 128, 2050 -> 771 49 / 59; 128 rows an
//     expert of 32 359 / 341
//   bf16, a few workgroups a CU, rows straight into LDS: 2x2 against 4x2: 1024 rows of 8
//     2048 -> 1250 11.4 / 13.7, -> 2600 17.1 / 19.9, -> 6000 34.5 / 30.9 (4x4)
//   bf16: 4x2 past the caches or through them g64 47 / 54, g256 79 / 78; 4x4 against 4x2
//     g256 76 / 78, g1024 142 / 167, g6400 684 / 801; of rows that are no whole 16 bytes
//     (2879 columns) 161 / 167 and 781 / 854, 4000 rows of 64 experts 511 -> 600 27.5 / 25.4
Fp4Choice choose(const Fp4GemmArgs &a, bool silu, bool bf16) {
  const int ne = a.E < a.R ? a.E : a.R, mean = a.R / ne;  // rows an expert, if all are hit
  const int H = silu ? 1 : 2;
  if (a.K < (bf16 ? 8 : 4)) {
    // (a thread for every 256th row at least, while that leaves at most 2^30 threads)
    const int most = (1 << 22) / ((a.N + 255) / 256 * ne);
    return {Fp4Kernel::kShort, std::min({mean, 256, most})};
  }
  if (mean <= 4) {
    const bool many = a.E > 1 && (long long)ne * ((a.NT + 2 * H - 1) / (2 * H)) >= 512;
    if (many && !bf16) return {Fp4Kernel::kTile4x1, 1};
    return {many ? Fp4Kernel::kStream4Once : Fp4Kernel::kStream2, a.R < 128 ? 1 : a.R < 256 ? a.R / 64 : 4};
  }
  if (workgroups(a, 16, 4) <= 320) return {Fp4Kernel::kSplit1x1, 1};
  const long long split = workgroups(a, bf16 ? 32 : 16, 4 * H);
  if (split <= (bf16 || a.NT <= 12 * H ? 288 : 384)) return {Fp4Kernel::kSplit2x2, 1};
  if (!bf16)
    return {mean <= 24 || workgroups(a, 32, 8 * H) < 512 ? Fp4Kernel::kTile4x1 : Fp4Kernel::kTile4x2, 1};
  if (a.K % 8 == 0 && (mean > 40 || a.E == 1) && split <= 1024) return {Fp4Kernel::kTile2x2, 1};
  if (mean >= 48 && workgroups(a, 64, 8 * H) >= 512)
    return {a.K % 8 == 0 ? Fp4Kernel::kTile4x4 : Fp4Kernel::kTile4x4Regs, 1};
  return {a.E > 1 && mean <= 40 ? Fp4Kernel::kTile4x2Once : Fp4Kernel::kTile4x2, 1};
}

template <bool SILU, typename DT>
hipError_t launch_t(const Fp4GemmArgs &a, Fp4Choice c, hipStream_t st) {
  constexpr int H = SILU ? 1 : 2;
  constexpr bool BF16 = sizeof(DT) == 2;
  switch (c.kernel) {
    case Fp4Kernel::kShort:
      return launch_kernel(k_fp4_short<SILU, DT>, dim3((a.N + 255) / 256, a.E < a.R ? a.E : a.R, c.groups), dim3(256),
                           0, st, a);
    case Fp4Kernel::kStream2: return stream_t<H, 8, false, SILU, DT>(a, st, c.groups);
    case Fp4Kernel::kSplit1x1: return tiled_t<SILU ? 2 : 1, 1, 4, false, false, SILU, DT>(a, st);
    case Fp4Kernel::kTile4x2: return tiled_t<4, 2, 1, false, false, SILU, DT>(a, st);
    case Fp4Kernel::kSplit2x2:
      // (float32: three parts in LDS, so fewer tokens)
      if constexpr (BF16) return tiled_t<2, 2, 4, false, false, SILU, DT>(a, st);
      else return tiled_t<4, 1, 4, false, false, SILU, DT>(a, st);
    case Fp4Kernel::kTile4x1:
      if constexpr (!BF16) return tiled_t<4, 1, 1, false, false, SILU, DT>(a, st);
      break;
    case Fp4Kernel::kStream4Once:
      if constexpr (BF16) return stream_t<2 * H, 4, true, SILU, DT>(a, st, c.groups);
      break;
    case Fp4Kernel::kTile2x2:
      if constexpr (BF16) return tiled_t<2, 2, 1, false, true, SILU, DT>(a, st);
      break;
    case Fp4Kernel::kTile4x2Once:
      if constexpr (BF16) return tiled_t<4, 2, 1, true, false, SILU, DT>(a, st);
      break;
    case Fp4Kernel::kTile4x4:
      if constexpr (BF16) return tiled_t<4, 4, 1, false, true, SILU, DT>(a, st);
      break;
    case Fp4Kernel::kTile4x4Regs:
      if constexpr (BF16) return tiled_t<4, 4, 1, false, false, SILU, DT>(a, st);
      break;
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
    if (bf16 ? kernel == Fp4Kernel::kTile4x1 : kernel >= Fp4Kernel::kStream4Once) continue;
    const hipError_t e = launch(a, silu, bf16, {kernel, 1}, nullptr);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moelora
