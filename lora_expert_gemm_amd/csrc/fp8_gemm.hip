// Grouped product of E4M3 rows and E4M3 weights with one float32 scale per
// block of 128 along the contraction:
//
//   out[m][n] = sum_b xs[b][m] ws[e][n / 128][b] sum_{k in block b} x[m][k] w[e][n][k]
//
// for the rows m of expert e, start[e] <= m < start[e + 1]; with SILU the
// weights are two matrices (gate, up) and out = SiLU(gate) * up.
//
// A block of 128 is exactly one v_mfma_f32_16x16x128_f8f6f4 of a 16 x 16
// output tile (weights on the row side, tokens on the column side), started
// from zero; its float32 result is multiplied by the two scales and added to
// the float32 accumulator, so the block sums never mix before they are
// scaled.  A lane's operand is 32 bytes of a row: any assignment of the
// block's 128 positions to lanes serves as long as both operands use the same.
//
// The FP8 forms of the matrix core add the eight products of a group after
// aligning them to the largest, and keep 13 bits below its leading one
// (measured: next to products of 2^16 that cancel, one of 2^3 survives in
// their group of eight and one of 2^2 does not, while between groups the sum
// is float32; the 16x16x32 form does the same).  A block sum S = sum |x w| is
// therefore off by at most 7 2^-13 S, and by 1.5e-5 of its own size on
// normal data: a hundredth of a bf16 rounding, though it moves one bf16 result
// in fifty to the neighbouring value.  The exact form widens the codes to bf16
// (exact) and lets four v_mfma_f32_16x16x32_bf16 form the block sum, whose
// products and float32 sum measured within 2^-20 of the largest product.  It is
// taken for float32 results, and for the 16-row streamed kernel whatever the
// type, where it costs next to nothing (16-token decode 60.1 -> 60.4 us, one row
// 9.84 -> 10.0).  bf16 results of the others take the FP8 form: the exact one
// costs the streamed kernel of 32 rows up to 11 %, tiles 5 to 55 % (64 tokens of
// the 32 experts 81 -> 89 us, 512 dense rows 33 -> 52), the 25600-row gate_up
// product nearly twice the time.
//
// Two kernels.  k_fp8_stream: few rows an expert, bound by the weights'
// bytes.  k_fp8_tiled: many rows, bound by the matrix cores.
#include "common.h"
#include "grouped.h"
#include "kernels.h"
#include "ops.h"

namespace moelora {

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// One block of a 16 x 16 tile, from zero: lane l supplies row l % 16 of each
// operand; the result has weight rows 4 (l / 16) + v, token l % 16.  Operand
// is what a lane's 32 codes become: themselves, or 32 bf16 values.
template <bool EXACT> struct Block;
template <> struct Block<false> {
  struct Operand {
    u32x4_t lo, hi;
  };
  __device__ __forceinline__ static Operand load(u32x4_t lo, u32x4_t hi) { return {lo, hi}; }
  __device__ __forceinline__ static f32x4_t mma(const Operand &a, const Operand &b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        __builtin_bit_cast(i32x8_t, a), __builtin_bit_cast(i32x8_t, b), f32x4_t{0, 0, 0, 0}, 0, 0, 0, 0,
        0, 0);  // (scale operands of zero: the form without scales)
  }
};
template <> struct Block<true> {
  struct Operand {
    u32x4_t q[4];
  };
  __device__ __forceinline__ static Operand load(u32x4_t lo, u32x4_t hi) {
    return {{e4m3x8_to_bf16(lo[0], lo[1]), e4m3x8_to_bf16(lo[2], lo[3]), e4m3x8_to_bf16(hi[0], hi[1]),
             e4m3x8_to_bf16(hi[2], hi[3])}};
  }
  __device__ __forceinline__ static f32x4_t mma(const Operand &a, const Operand &b) {
    f32x4_t c = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) Mma<uint16_t>::step(c, a.q[i], b.q[i]);
    return c;
  }
};

// A block sum's two scales are multiplied with each other first: one multiply
// for a token and a weight block where scaling the sum twice would take one an
// accumulator.  Where that product overflows though neither scale is infinite,
// the sum (of finite codes: 0, or between 2^-18 and 2^25) takes the larger scale
// first and the other in the multiply-add, so a block of zeros stays zero and a
// small sum finite.  A product below 2^-126 is rounded by up to 2^-150, which
// moves its block by up to 2^-125; scaling those twice as well would make up for
// it, but rows of zeros (scale 2^-126) are among them, and a few of those took
// the 25600-row gate_up product from 480 to 640 us.  Looking for overflow costs
// that product 1.7 % (455 -> 463 us), 512 dense rows 1 %, the streamed kernel
// nothing.
__device__ __forceinline__ bool overflows(float product) {
  return __builtin_amdgcn_classf(product, 0x204);  // -inf, +inf
}
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
// s: the product of a and b, or the smaller of them where that overflows, with
// the larger in first (1 for the lanes that need nothing: they stay bit for bit
// what they are without such a neighbour).
__device__ __forceinline__ void split_scale(float &s, float &first, float a, float b) {
  const bool odd = overflows(s), a_first = fabsf(a) > fabsf(b);
  first = odd ? a_first ? a : b : 1.f;
  s = odd ? a_first ? b : a : s;
}

// ---------------------------------------------------------------- few rows
//
// A workgroup owns 16 NT weight rows (of each half) of one expert and up to
// 16 TG of its tokens at a time (every gridDim.z-th group); its four waves take every fourth block of
// the contraction and add their sums through LDS in wave order, so that a
// narrow product still fills the chip.  Each wave streams its weights through
// an LDS ring of its own, S blocks deep, in whole 128-byte lines (8 lanes a
// line): loaded straight into operand registers, 16 rows at 64 bytes an
// instruction, the address unit and not HBM set the pace.  Tokens, few and
// shared by all workgroups, come from cache into registers.  Bound by the
// weights' bytes: the 16-token decode step of 32 experts (392 MB of 23 experts
// hit) takes 58-64 us by card, 6.1-6.8 TB/s (77 us with the weights straight into
// registers; 75 us with a ring of 4 blocks, whose 64 KB leave two workgroups
// on a CU where 2 blocks leave four), one row of 4096 -> 11008 (45 MB) 9.8 us.
constexpr int kSWaves = 4;
constexpr int kSThreads = kSWaves * kWave;

// LDS byte offset of 16-byte chunk c of a 128-byte row: 16 consecutive rows
// read at one chunk fall on 16 distinct bank groups.
__device__ __forceinline__ int lds_off(int row, int c) {
  return row * 128 + ((c ^ ((row >> 1) & 7)) << 4);
}

template <int NT, int TG, int S, bool ONCE, bool SILU, typename OT>
__global__ __launch_bounds__(kSThreads) void k_fp8_stream(Fp8GemmArgs a) {
  constexpr int HV = SILU ? 2 : 1, A = HV * NT;
  constexpr int SLOT = A * 16 * 128;
  typedef Block<sizeof(OT) == 4 || TG == 1> B;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ f32x4_t red[kSWaves][A * TG][kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int l16 = lane & 15, g = lane >> 4;
  // the expert: blockIdx.y itself, or the blockIdx.y-th that has rows
  int e, lo, hi;
  if (!find_expert(a, blockIdx.y, e, lo, hi)) return;
  const int KB = a.KB, n0 = blockIdx.x * NT * 16, cols = min(NT * 16, a.N - n0);
  const size_t mat = (size_t)e * HV;
  const uint8_t *wbase[2] = {a.w + (mat * a.N + n0) * a.P, a.w + ((mat + HV - 1) * a.N + n0) * a.P};
  uint32_t woff[8];
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) {
    const int r = 8 * j + (lane >> 3);
    woff[j] = (uint32_t)(r * a.P) + 16 * ((lane & 7) ^ ((r >> 1) & 7));
  }
  // weight scales 64 blocks at a time, one a lane (the workgroup's columns lie
  // in one block of 128)
  static_assert(NT <= 4 && 16 % S == 0, "");
  const float *wsp = a.ws + (mat * a.NB + n0 / 128) * KB;
  float ws[HV];
  unsigned char *const ring = smem + wave * (S * SLOT);

  for (int m0 = lo + blockIdx.z * 16 * TG; m0 < hi; m0 += gridDim.z * 16 * TG) {
    f32x4_t acc[A][TG];
#pragma unroll
    for (int i = 0; i < A; ++i)
#pragma unroll
      for (int t = 0; t < TG; ++t) acc[i][t] = f32x4_t{0, 0, 0, 0};
    const uint8_t *xp[TG];
    int xr[TG];
#pragma unroll
    for (int t = 0; t < TG; ++t) {
      xr[t] = min(m0 + 16 * t + l16, hi - 1);  // (rows past the last repeat it and are dropped)
      xp[t] = a.x + (size_t)xr[t] * a.P + g * 16;
    }
    u32x4_t x0[S][TG], x1[S][TG];
    float sx[S][TG];
    // block b into slot u: weights by direct loads to LDS (past the last
    // block from an empty resource: they fetch nothing), tokens into registers
    auto issue = [&](int u, int b) {
#pragma unroll
      for (int h = 0; h < HV; ++h) {
        const __amdgpu_buffer_rsrc_t res = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t *>(wbase[h]), (short)0, b < KB ? (int)(cols * a.P) : 0, kBufferWord3);
#pragma unroll
        for (int j = 0; j < 2 * NT; ++j)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(
              res, (__attribute__((address_space(3))) void *)(ring + u * SLOT + (h * NT * 16 + 8 * j) * 128),
              16, woff[j], b * 128, 0, ONCE ? kCpolNonTemporal : 0);
      }
      const int bc = min(b, KB - 1);
#pragma unroll
      for (int t = 0; t < TG; ++t) {
        x0[u][t] = *reinterpret_cast<const u32x4_t *>(xp[t] + (size_t)bc * 128);
        x1[u][t] = *reinterpret_cast<const u32x4_t *>(xp[t] + (size_t)bc * 128 + 64);
        sx[u][t] = a.xs[(size_t)bc * a.R + xr[t]];
      }
    };
#pragma unroll
    for (int u = 0; u < S; ++u) issue(u, wave + u * kSWaves);
    for (int b0 = wave; b0 < KB; b0 += kSWaves * S) {
      if (b0 % kWave == wave) {
#pragma unroll
        for (int h = 0; h < HV; ++h)
          ws[h] = wsp[(size_t)h * a.NB * KB + min(b0 - wave + lane, KB - 1)];
      }
#pragma unroll
      for (int u = 0; u < S; ++u) {
        const int b = b0 + u * kSWaves;
        // loads return in order: no more than the S - 1 later blocks' weight
        // loads may be in flight when this block is read
        __builtin_amdgcn_s_waitcnt(wait_vmcnt((S - 1) * 2 * A));
        __builtin_amdgcn_sched_barrier(0);
        if (b < KB) {
          const unsigned char *st = ring + u * SLOT;
          float sw[HV];
#pragma unroll
          for (int h = 0; h < HV; ++h)
            sw[h] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ws[h]), b % kWave));
          typename B::Operand w[A];
#pragma unroll
          for (int i = 0; i < A; ++i)
            w[i] = B::load(*reinterpret_cast<const u32x4_t *>(st + lds_off(16 * i + l16, g)),
                           *reinterpret_cast<const u32x4_t *>(st + lds_off(16 * i + l16, g + 4)));
#pragma unroll
          for (int t = 0; t < TG; ++t) {
            const typename B::Operand x = B::load(x0[u][t], x1[u][t]);
            f32x4_t p[A];
#pragma unroll
            for (int i = 0; i < A; ++i) p[i] = B::mma(w[i], x);
            float s[HV], first[HV];
            bool odd = false;
#pragma unroll
            for (int h = 0; h < HV; ++h) {
              s[h] = sx[u][t] * sw[h];
              odd |= overflows(s[h]);
            }
            if (__builtin_expect(__any(odd), 0)) {
#pragma unroll
              for (int h = 0; h < HV; ++h) split_scale(s[h], first[h], sx[u][t], sw[h]);
#pragma unroll
              for (int i = 0; i < A; ++i) p[i] *= first[i / NT];
            }
#pragma unroll
            for (int i = 0; i < A; ++i)
#pragma unroll
              for (int v = 0; v < 4; ++v) acc[i][t][v] = fmaf(s[i / NT], p[i][v], acc[i][t][v]);
          }
        }
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the slot is read out
        issue(u, b + kSWaves * S);
      }
    }
    __builtin_amdgcn_s_waitcnt(0x0f70);  // no load outlives its slot
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
      const int m = m0 + 16 * t + l16, n = n0 + 16 * i + 4 * g;
      if (m < hi && n < a.N) {
        float o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = SILU ? silu_mul<sizeof(OT) == 4>(v[0][c], v[HV - 1][c]) : v[0][c];
        store4<OT>(static_cast<OT *>(a.out) + (size_t)m * a.N, n, a.N, o);
      }
    }
    __syncthreads();
  }
}

// --------------------------------------------------------------- many rows
//
// 16 TT token rows x 64 WT weight rows (SILU: half gate, half up) a workgroup
// of 4 waves, two workgroups or more per CU.  A wave owns 16 WT weight rows
// against all the tokens.  Everything arrives in slabs of one block of 128,
// one 128-byte line a row, fetched by 8 lanes straight into LDS: the tokens
// and their scales into two stages that the waves share (loaded one slab
// ahead, one barrier a slab), the weights, which no other wave reads, into a
// place of the wave's own, from which they go on to registers half a slab
// before they are needed, so that the next slab's can be on their way with no
// barrier.  A row's 16-byte chunk c sits at chunk c ^ ((row / 2) % 8) of its
// LDS row, so the 16 rows that 16 lanes read at one chunk fall on 16 distinct
// bank groups.  Rows past the expert's last, and weight rows past N, lie past
// their buffer resource's end: their loads fetch nothing, and their outputs
// are dropped.
//
// What led here, for the 25600-row gate_up product of 32 experts (849 GFLOP;
// the same card's library product of plain E4M3 without block scales runs at
// 2.6-2.75 PFLOP/s): 128 x 512 tiles of 8 waves, everything through two shared
// stages, 672 us; weights straight into registers, two 4-wave workgroups per
// CU, 574 us (the address unit takes 16 rows at 64 bytes an instruction);
// weights through the wave's own LDS in whole lines, 523 us where the step
// before took 671 (another card); block sums scaled four MFMAs after they were
// formed, 484 us; the shorter epilogue, 452-474 us by card, and the check for
// overflowing scales, 460-485: 1.75-1.85 PFLOP/s.
// The matrix cores are busy 53 % of the cycles, at 1.8 GHz under the card's
// power limit.  Without its loads the loop keeps them 68 % busy, and leaving
// out the waits for the loads changes nothing: the loads' own passage
// (1.3 GB from beyond L2, 77 % L2 hits) and the one multiply-add an
// accumulator and block that the scales cost bound it now.
constexpr int kGWaves = 4, kGThreads = kGWaves * kWave;
constexpr int kGSlots = 2;              // stages of tokens

template <int WT, int TT, bool ONCE, bool SILU, typename OT>
__global__ __launch_bounds__(kGThreads, sizeof(OT) == 2 && WT * TT <= 8 ? 3 : 2) void k_fp8_tiled(
    Fp8GemmArgs a, int ncols) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int HV = SILU ? 2 : 1, WH = WT / HV;        // weight tiles of a half
  constexpr int WC = 16 * WH, COLS = kGWaves * WC;      // columns a wave, a workgroup
  constexpr int GM = 16 * TT, STAGE = GM * 128 + 512;
  constexpr int XL = GM / 8 / kGWaves;  // token loads a wave and slab
  typedef Block<sizeof(OT) == 4> B;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int l16 = lane & 15, g = lane >> 4;
  const RowTile rt = find_tile(a, GM, ncols, blockIdx.x);
  if (rt.e < 0) return;
  const int n0 = rt.nt * COLS, rows = min(GM, rt.hi - rt.m0), cols = min(COLS, a.N - n0);
  const size_t P = a.P;
  const int KB = a.KB;

  // Buffer resources of the tile; slabs past the last get an empty one, so
  // the loop issues its loads unconditionally and they fetch nothing.
  const size_t mat = (size_t)rt.e * HV;
  const uint8_t *wbase[2] = {a.w + (mat * a.N + n0) * P, a.w + ((mat + HV - 1) * a.N + n0) * P};
  auto resource = [&](const void *base, int bytes, int b) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, b < KB ? bytes : 0,
                                             kBufferWord3);
  };
  // load plans: a wave instruction fills 8 LDS rows (1 KB), lane i bringing
  // the chunk that lds_off places at byte 16 i of the group.  The wave's
  // 16 WT weight rows are WC of each half.
  uint32_t woff[16];
#pragma unroll
  for (int j = 0; j < WC / 8; ++j) {
    const int r = 8 * j + (lane >> 3);
    woff[j] = (uint32_t)((WC * wave + r) * P) + 16 * ((lane & 7) ^ ((r >> 1) & 7));
  }
  uint32_t xoff[4];
#pragma unroll
  for (int j = 0; j < XL; ++j) {
    const int r = 8 * (XL * wave + j) + (lane >> 3);
    xoff[j] = (uint32_t)(r * P) + 16 * ((lane & 7) ^ ((r >> 1) & 7));
  }
  unsigned char *const wst = smem + kGSlots * STAGE + wave * (WT * 16 * 128);
  struct Weights {
    typename Block<false>::Operand v[WT];
  };
  auto issue_w = [&](int b) {
#pragma unroll
    for (int j = 0; j < 2 * WT; ++j) {
      const __amdgpu_buffer_rsrc_t res = resource(wbase[j * 8 / WC], (int)(cols * P), b);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          res, (__attribute__((address_space(3))) void *)(wst + 8 * j * 128), 16, woff[j % (WC / 8)],
          b * 128, 0, ONCE ? kCpolNonTemporal : 0);
    }
  };
  auto read_w = [&](Weights &w) {
#pragma unroll
    for (int i = 0; i < WT; ++i)
      w.v[i] = {*reinterpret_cast<const u32x4_t *>(wst + lds_off(16 * i + l16, g)),
                *reinterpret_cast<const u32x4_t *>(wst + lds_off(16 * i + l16, g + 4))};
  };
  // tokens and their scales (64 a wave, twice over) of slab b
  auto issue_x = [&](int b) {
    unsigned char *st = smem + b % kGSlots * STAGE;
    const __amdgpu_buffer_rsrc_t xres = resource(a.x + (size_t)rt.m0 * P, (int)(rows * P), b);
#pragma unroll
    for (int j = 0; j < XL; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          xres, (__attribute__((address_space(3))) void *)(st + 8 * (XL * wave + j) * 128), 16, xoff[j],
          b * 128, 0, 0);
    const __amdgpu_buffer_rsrc_t sres = resource(a.xs + (size_t)b * a.R + rt.m0, rows * 4, b);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        sres, (__attribute__((address_space(3))) void *)(st + GM * 128 + 256 * (wave & 1)), 4,
        256 * (wave & 1) + 4 * lane, 0, 0, 0);
  };
  // scales of the wave's weight block: 64 slabs at a time, one a lane (the
  // wave's WC columns lie in one block of 128)
  const float *wsp = a.ws + (mat * a.NB + min((n0 + WC * wave) / 128, a.NB - 1)) * KB;
  float ws[HV];

  constexpr int SL = (GM + kWave - 1) / kWave;  // tokens' scales of a slab, a lane
  int sxat[SL];  // ... and where it lies in a stage (rows past the last: the last's)
#pragma unroll
  for (int q = 0; q < SL; ++q) sxat[q] = GM * 128 + 4 * min(kWave * q + lane, rows - 1);

  f32x4_t acc[WT][TT];
#pragma unroll
  for (int i = 0; i < WT; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[i][t] = f32x4_t{0, 0, 0, 0};

  // block sums not yet added, and their scales
  f32x4_t p[WT];
  float s[HV];
#pragma unroll
  for (int i = 0; i < WT; ++i) p[i] = f32x4_t{0, 0, 0, 0};
#pragma unroll
  for (int h = 0; h < HV; ++h) s[h] = 0.f;
  auto add = [&](int i, int t) {
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[i][t][v] = fmaf(s[SILU ? i / WH : 0], p[i][v], acc[i][t][v]);
    // (or the compiler sinks the multiply-adds past the branches on large scales
    // to the slab's end, and keeps every group's block sums until there)
    asm volatile("" : "+v"(acc[i][t]));
  };

  // Slab b with its weights in `w`; reads slab b + 1's into `wn` half way.
  // The waits count this wave's own loads in their order of issue: tokens of
  // b + 1 (XL + 1 loads, top of slab b), weights of b + 2 (2 WT loads, middle of
  // slab b); nothing moves across the barrier or the waits.
  auto step = [&](int b, const Weights &w, Weights &wn) {
    // tokens of b landed (weights of b + 1 may not have) and this wave's reads
    // of slab b - 1 done (lgkmcnt(0)) ...
    __builtin_amdgcn_s_waitcnt(wait_vmcnt(2 * WT) & ~0x0f00);
    __builtin_amdgcn_s_barrier();  // ... for every wave
    if (b % kWave == 0) {
#pragma unroll
      for (int h = 0; h < HV; ++h) ws[h] = wsp[(size_t)h * a.NB * KB + min(b + lane, KB - 1)];
      // (waited for here: or every slab waits for a load that it may have made,
      // and with it for the weights of the slab after)
#pragma unroll
      for (int h = 0; h < HV; ++h) asm volatile("" : "+v"(ws[h]));
    }
    issue_x(b + 1);
    const unsigned char *st = smem + b % kGSlots * STAGE;
    const float *sx = reinterpret_cast<const float *>(st + GM * 128);
    float sw[HV];
#pragma unroll
    for (int h = 0; h < HV; ++h)
      sw[h] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ws[h]), b % kWave));
    typename B::Operand wo[WT];
#pragma unroll
    for (int i = 0; i < WT; ++i) wo[i] = B::load(w.v[i].lo, w.v[i].hi);
    // token fragments one group ahead of their MFMAs; the scheduling barrier
    // keeps the compiler from reading all groups at once (registers)
    auto read_x = [&](int t, u32x4_t &lo, u32x4_t &hi) {
      const int r = 16 * t + l16;
      lo = *reinterpret_cast<const u32x4_t *>(st + lds_off(r, g));
      hi = *reinterpret_cast<const u32x4_t *>(st + lds_off(r, g + 4));
    };
    u32x4_t xlo[2], xhi[2];
    read_x(0, xlo[0], xhi[0]);
    // whether any two scales of the slab overflow, all tokens and halves at once
    // (by the largest)
    float sxq[SL];
#pragma unroll
    for (int q = 0; q < SL; ++q) sxq[q] = *reinterpret_cast<const float *>(st + sxat[q]);
    unsigned long long odd = 0;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      if (t + 1 < TT) read_x(t + 1, xlo[(t + 1) & 1], xhi[(t + 1) & 1]);
      const float sxt = sx[16 * t + l16];
      const typename B::Operand x = B::load(xlo[t & 1], xhi[t & 1]);
      // a block sum is scaled and added just before its register takes the
      // next group's: WT MFMAs later, so nothing waits for the matrix core
#pragma unroll
      for (int i = 0; i < WT; ++i) {
        add(i, t == 0 ? TT - 1 : t - 1);
        p[i] = B::mma(wo[i], x);
        __builtin_amdgcn_sched_barrier(0);
        if (t == 0 && i == WT - 1) {
#pragma unroll
          for (int q = 0; q < SL; ++q) asm volatile("" : "+v"(sxq[q]));  // (here, behind the MFMA)
          uint32_t mx = magnitude(sxq[0]), wmx = magnitude(sw[0]);
          if constexpr (SL > 1) mx = max(mx, magnitude(sxq[SL - 1]));
          if constexpr (HV > 1) wmx = max(wmx, magnitude(sw[HV - 1]));
          const float most = __uint_as_float(mx) * __uint_as_float(wmx);
          odd = __builtin_amdgcn_ballot_w64(!(most <= __FLT_MAX__));  // (NaN too)
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int h = 0; h < HV; ++h) s[h] = sxt * sw[h];
      asm volatile("" : "+s"(odd));  // (one scalar comparison a group, not a lane mask kept)
      if (__builtin_expect(odd != 0, 0)) {
        float first[HV];
#pragma unroll
        for (int h = 0; h < HV; ++h) split_scale(s[h], first[h], sxt, sw[h]);
#pragma unroll
        for (int i = 0; i < WT; ++i) p[i] *= first[SILU ? i / WH : 0];
      }
      __builtin_amdgcn_sched_barrier(0);
      if (t == TT / 2 - 1) {
        __builtin_amdgcn_s_waitcnt(wait_vmcnt(XL + 1));  // weights of b + 1 landed
        read_w(wn);
      }
      if (t == TT / 2) {
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): read out, their place is free
        issue_w(b + 2);
      }
    }
  };

  Weights wa, wb;
  issue_w(0);
  __builtin_amdgcn_s_waitcnt(0x0f70);
  read_w(wa);
  __builtin_amdgcn_s_waitcnt(0xc07f);
  issue_x(0);
  issue_w(1);
  int b = 0;
  for (; b + 1 < KB; b += 2) {
    step(b, wa, wb);
    step(b + 1, wb, wa);
  }
  if (b < KB) step(b, wa, wb);
#pragma unroll
  for (int i = 0; i < WT; ++i) add(i, TT - 1);
  __builtin_amdgcn_s_waitcnt(0x0f70);  // no load of this workgroup outlives it

#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int m = 16 * t + l16;
    if (m >= rows) continue;
    OT *row = static_cast<OT *>(a.out) + (size_t)(rt.m0 + m) * a.N;
#pragma unroll
    for (int i = 0; i < WH; ++i) {
      const int n = n0 + WC * wave + 16 * i + 4 * g;
      if (n >= a.N) continue;
      float o[4];
#pragma unroll
      for (int v = 0; v < 4; ++v)
        o[v] = SILU ? silu_mul<sizeof(OT) == 4>(acc[i][t][v], acc[(i + WH) % WT][t][v]) : acc[i][t][v];
      store4<OT>(row, n, a.N, o);
    }
  }
}

template <int NT, int TG, int S, bool ONCE, bool SILU, typename OT>
hipError_t stream_t(const Fp8GemmArgs &a, hipStream_t st, int splits = 1) {
  constexpr int LDS = kSWaves * S * NT * (SILU ? 2 : 1) * 16 * 128;
  auto kern = k_fp8_stream<NT, TG, S, ONCE, SILU, OT>;
  hipError_t err = hipFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
  if (err != hipSuccess) return err;
  return launch_kernel(kern, dim3((a.N + 16 * NT - 1) / (16 * NT), a.E < a.R ? a.E : a.R, splits),
                       dim3(kSThreads), LDS, st, a);
}

template <int WT, int TT, bool ONCE, bool SILU, typename OT>
hipError_t tiled_t(const Fp8GemmArgs &a, hipStream_t st) {
  constexpr int COLS = kGWaves * 16 * WT / (SILU ? 2 : 1), GM = 16 * TT;
  constexpr int LDS = kGSlots * (GM * 128 + 512) + kGWaves * 16 * WT * 128;
  auto kern = k_fp8_tiled<WT, TT, ONCE, SILU, OT>;
  hipError_t err = hipFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
  if (err != hipSuccess) return err;
  const int ncols = (a.N + COLS - 1) / COLS;
  const int ne = a.E < a.R ? a.E : a.R;
  const int tiles = (int)(((long long)a.R + (long long)ne * (GM - 1)) / GM);
  return launch_kernel(kern, dim3(round_up8(tiles * ncols)), dim3(kGThreads), LDS, st, a, ncols);
}

// Most workgroups a tiled launch can hold: row tiles of GM rows (each expert's
// last one short) times column tiles.
long long tiled_wgs(const Fp8GemmArgs &a, bool silu, int WT, int TT) {
  const long long GM = 16 * TT, cols = kGWaves * 16 * WT / (silu ? 2 : 1);
  const long long ne = a.E < a.R ? a.E : a.R;
  return (a.R + ne * (GM - 1)) / GM * ((a.N + cols - 1) / cols);
}

// Which kernel, by the mean rows of an expert and by how many workgroups a
// tile leaves (two of 128 tokens x 256 weight rows fit a CU: 512 on the
// chip).  us on one card, E = 32, top-4, 2880 -> 2 x 2880 with SILU ("g", by
// tokens), and dense 4096 -> 11008 ("d", by rows):
//            few rows      tiles: WT x TT, weights through the caches
//            1x16  2x16    2x2   2x4   2x8   4x8
//   g32      73    81      87    89    89   106
//   g64      97    93      97    94    97   110
//   g256    257   184     115   109   109   117
//   g512    481   312     151   126   121   119
//   g1024   944   585     215   169   147   142
//   d16      13    14      18    18    22    32
//   d32      22    16      18    18    22    32
//   d64      42    29      18    19    23    33
//   d512    328   217      49    34    35    37
//   d1024   663   435      90    66    53    58
Fp8Choice choose(const Fp8GemmArgs &a, bool silu, bool bf16) {
  const int mean = a.R / (a.E < a.R ? a.E : a.R);  // rows an expert, if all are hit
  const int NT = silu ? 1 : 2;  // 32 weight rows a workgroup either way
  // (several experts: some have twice the mean, and pass their weights twice; an
  // expert with many times the mean passes them once every 16 rows, one after
  // the other: 896 rows of one of 128 experts, 2880 -> 2 x 2880, 340-360 us, spread
  // evenly 332.  One expert's weights may still lie in the last-level cache,
  // several are streamed past it: a single row of 4096 -> 11008 9.9 us against
  // 10.6, the 16-token decode 59 us against 66)
  // Short rows leave the waves that share K there without blocks of their own
  // and each workgroup little but its start and end; a tile has fewer
  // workgroups, each with more to write.  us, this and a tile's, 64 experts,
  // 128 rows, -> 2 x 2880 with SILU by K: 128 23.9 / 11.9, 512 35.7 / 25.1, 768
  // 40.0 / 35.1, 1024 46.3 / 43.6 (float32 768 40.9 / 37.2, 256 rows -> 2880
  // 26.8 / 28.4).  With few tiles the longer chain of a tile shows: 8 rows of
  // 512 -> 2880 5.4 / 6.5 (184 tiles), 128 rows -> 768 6.9 / 6.8 (396).
  if (a.E > 1 && mean <= 7) {
    if (a.KB <= (bf16 ? 6 : 5) && tiled_wgs(a, silu, 2, 2) >= 100LL * a.KB)
      return {Fp8Kernel::kTile2x2Once, 1};
    return {Fp8Kernel::kStream1Once, 1};
  }
  // So little work that tiles would leave most of the chip idle: an expert's
  // row groups go to workgroups of their own, with the weights from cache.
  // One expert, us, a tile's and this: 64 x 4096 -> 2048 12.4 / 6.7, 256 x 4096 ->
  // 1024 16.2 / 8.4, 1000 x 8000 -> 200 27.9 / 14.2, 128 x 2880 -> 2880 13.1 / 12.2,
  // twice that 13.4 / 16.6.  Eight experts, 4096 ->, by rows an expert and
  // columns: 8, 256 23.5 / 6.5; 8, 2048 25.7 / 14.8; 16, 2048 25.7 / 17.8; 24, 4096
  // 32.3 / 34.8; 32, 256 16.5 / 8.0; 48, 1024 16.9 / 19.4; 32 experts: 8, 256 24.3 /
  // 13.2; 32, 256 17.2 / 26.9.  A tile walks the contraction alone, a slab after
  // the other, while the streamed kernel's four waves share it, so the longer
  // it is the more work may go there: of 45 sizes past 24 blocks with up to 320
  // workgroups (8 to 40 experts of 32 to 150 rows, K 3300 to 8192, either type)
  // 43 took 0.43 to 0.99 of a tile's time and two 1.05; of eleven sizes of 12
  // blocks eight took 1.03 to 1.33.
  // Fuller experts than the mean take more groups: a
  // launch has room for twice the mean and more where that costs little,
  // and a workgroup goes on to the next group if that is not enough.
  const int ne = a.E < a.R ? a.E : a.R, cols = (a.N + 16 * NT - 1) / (16 * NT);
  auto wgs = [&](int rows) { return cols * ((a.R + (long long)ne * (rows - 1)) / rows); };
  auto groups = [&](int rows) {
    const int all = (a.R + rows - 1) / rows, twice = (2 * mean + rows - 1) / rows + 1;
    const long long room = 1024 / ((long long)cols * ne);
    return a.E == 1 || all < twice ? all : room > all ? all : room > twice ? (int)room : twice;
  };
  if ((a.E == 1 && a.R <= 16) || wgs(16) <= (a.E == 1 ? 256 : 192))
    return {Fp8Kernel::kStream1, groups(16)};
  if ((a.E == 1 && a.R <= 32) || wgs(32) <= (a.E == 1 ? 384 : mean <= 24 ? 960 : a.KB > 24 ? 320 : 192))
    return {Fp8Kernel::kStream2, groups(32)};
  if (bf16) {
    if (mean >= 56 && tiled_wgs(a, silu, 4, 8) >= 512) return {Fp8Kernel::kTile4x8, 1};
    if (mean >= 96 && tiled_wgs(a, silu, 2, 8) >= 512) return {Fp8Kernel::kTile2x8, 1};
  } else {
    // float32 results: widened operands leave registers for 64 tokens (the
    // 25600-row gate_up 866 us against 919 with 2x4, g1024 201 against 198; since
    // then 862-905 by card with the longer SiLU and the check for overflowing scales)
    if (mean >= 192 && tiled_wgs(a, silu, 4, 4) >= 512) return {Fp8Kernel::kTile4x4, 1};
  }
  // Where an expert's rows mostly fit one row tile its weights are read once:
  // past the caches then (16-row experts of 128: 78 -> 70 us, g64 94 -> 83,
  // g256 109 -> 105; with seven row tiles an expert, 471 -> 535).  Not for one
  // expert, whose weights may still lie in the last-level cache (d64 18 -> 24).
  // float32 results widen every row of a tile, padding too, so 64-row tiles
  // want more than 24 rows an expert: time of 2x4 over 2x2 for 32 to 128 experts,
  // 2050 -> 771, 2880 -> 2880 and 1024 -> 4096, 9 rows 1.01-1.32, 16 0.95-1.17, 24
  // 0.88-1.04, 28 0.86-1.02, 40 0.83-0.99 (32 experts -> 771 1.19).
  if (tiled_wgs(a, silu, 2, 4) >= 160 && (bf16 || mean > 24)) {
    if (a.E > 1 && mean <= 40) return {Fp8Kernel::kTile2x4Once, 1};
    return {Fp8Kernel::kTile2x4, 1};
  }
  if (a.E > 1 && mean <= 24) return {Fp8Kernel::kTile2x2Once, 1};
  return {Fp8Kernel::kTile2x2, 1};
}

template <bool SILU, typename OT>
hipError_t launch_t(const Fp8GemmArgs &a, Fp8Choice c, hipStream_t st) {
  constexpr int NT = SILU ? 1 : 2;
  switch (c.kernel) {
    case Fp8Kernel::kStream1Once: return stream_t<NT, 1, 2, true, SILU, OT>(a, st, c.groups);
    case Fp8Kernel::kStream1: return stream_t<NT, 1, 2, false, SILU, OT>(a, st, c.groups);
    case Fp8Kernel::kStream2: return stream_t<NT, 2, 2, false, SILU, OT>(a, st, c.groups);
    case Fp8Kernel::kTile2x2Once: return tiled_t<2, 2, true, SILU, OT>(a, st);
    case Fp8Kernel::kTile2x2: return tiled_t<2, 2, false, SILU, OT>(a, st);
    case Fp8Kernel::kTile2x4Once: return tiled_t<2, 4, true, SILU, OT>(a, st);
    case Fp8Kernel::kTile2x4: return tiled_t<2, 4, false, SILU, OT>(a, st);
    case Fp8Kernel::kTile2x8:
      if constexpr (sizeof(OT) == 2) return tiled_t<2, 8, false, SILU, OT>(a, st);
      break;
    case Fp8Kernel::kTile4x8:
      if constexpr (sizeof(OT) == 2) return tiled_t<4, 8, false, SILU, OT>(a, st);
      break;
    case Fp8Kernel::kTile4x4:
      if constexpr (sizeof(OT) == 4) return tiled_t<4, 4, false, SILU, OT>(a, st);
      break;
  }
  return hipErrorInvalidValue;
}

hipError_t launch(const Fp8GemmArgs &a, bool silu, bool bf16, Fp8Choice c, hipStream_t st) {
  if (silu) return bf16 ? launch_t<true, uint16_t>(a, c, st) : launch_t<true, float>(a, c, st);
  return bf16 ? launch_t<false, uint16_t>(a, c, st) : launch_t<false, float>(a, c, st);
}

}  // namespace

Fp8Choice choose_fp8_gemm(const Fp8GemmArgs &a, bool silu, bool bf16) { return choose(a, silu, bf16); }

hipError_t launch_fp8_gemm(const Fp8GemmArgs &a, bool silu, bool bf16, hipStream_t st) {
  return launch(a, silu, bf16, choose(a, silu, bf16), st);
}

hipError_t resolve_fp8_gemm(bool silu, bool bf16) {
  Fp8GemmArgs a{};
  a.R = a.N = a.K = a.E = a.KB = a.NB = 1, a.P = 128;
  for (Fp8Kernel k : {Fp8Kernel::kStream1Once, Fp8Kernel::kStream1, Fp8Kernel::kStream2, Fp8Kernel::kTile2x2Once,
                      Fp8Kernel::kTile2x2, Fp8Kernel::kTile2x4Once, Fp8Kernel::kTile2x4, Fp8Kernel::kTile2x8,
                      Fp8Kernel::kTile4x8, Fp8Kernel::kTile4x4}) {
    if (bf16 ? k == Fp8Kernel::kTile4x4 : k == Fp8Kernel::kTile2x8 || k == Fp8Kernel::kTile4x8) continue;
    const hipError_t e = launch(a, silu, bf16, {k, 1}, nullptr);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moelora
