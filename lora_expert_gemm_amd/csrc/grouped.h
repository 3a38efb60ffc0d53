// What the grouped products share: the ranges of the experts' rows, the items
// of a tiled launch, SiLU(gate) * up and the stores of results.
#pragma once

#include "common.h"

namespace moelora {

// Four consecutive outputs of a row, n .. n + 3 of N: one store, which needs
// no alignment beyond the element's here, or the row's last few by themselves.
template <typename OT>
__device__ __forceinline__ void store4(OT *row, int n, int N, const float *v) {
  typedef uint32_t words __attribute__((ext_vector_type(sizeof(OT))));
  typedef words mem __attribute__((aligned(2)));
  OT o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(OT) == 2) o[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);  // nearest even
    else o[i] = v[i];
  }
  if (n + 4 <= N) {
    *reinterpret_cast<mem *>(row + n) = __builtin_bit_cast(words, o);
  } else {
    for (int i = 0; i < 4; ++i)
      if (n + i < N) row[n + i] = o[i];
  }
}

// g / (1 + e^-g) u.  For bf16 results with the hardware's 2^x and 1 / x: the
// argument -log2(e) g is one rounded product, so the value is off by up to
// |g| 2^-23 of itself, and a sigmoid below 2^-126 counts as zero; with a
// correctly rounded division and exponential the epilogue was a third of the
// tiled kernel's vector instructions.  float32 results do not take that: there
// e^-|g| is the square of r = e^(-|g| / 2) = 2^y (1 + rest ln 2), with the
// rounding of y made good, and for g < 0 one r goes to each factor,
// (g r) / (1 + r r) (u r): nothing underflows before the result does, down to
// g = -174 (a sigmoid of 2^-251; below, zero).  25600 rows of gate_up in float32
// take 878 us with the short form, 895 with this, 905 with expf.
template <bool EXACT>
__device__ __forceinline__ float silu_mul(float g, float u) {
  if constexpr (EXACT) {
    constexpr float kLog2e = 0x1.715476p0f, kRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;  // log2(e) in two
    const float x = -0.5f * fminf(fabsf(g), 400.f), y = x * kLog2e;  // (finite: so is the rest)
    const float rest = fmaf(x, kRest, fmaf(x, kLog2e, -y));  // what the argument y lost
    const float p = __builtin_amdgcn_exp2f(y), r = fmaf(p, rest * kLn2, p);
    const float q = __builtin_amdgcn_rcpf(fmaf(r, r, 1.f));
    return g < 0.f ? g * r * q * (u * r) : g * q * u;
  } else {
    const float e = __builtin_amdgcn_exp2f(-1.44269504088896340736f * g);
    return g * __builtin_amdgcn_rcpf(1.f + e) * u;
  }
}

// s_waitcnt operand that waits for all but the n newest vector loads.
constexpr int wait_vmcnt(int n) { return 0x0f70 | (n & 15) | (n >> 4) << 14; }

// start[] entries are device data: clamped into [0, R].
__device__ __forceinline__ int row_bound(const int *start, int e, int R) {
  return min(max(start[e], 0), R);
}

// The expert of workgroup row `want` (of min(E, R)) and its rows [lo, hi): expert
// `want` itself or, where there are more experts than rows, the want-th that has
// any.  False: none.  Looked up by the whole wave.
template <typename Args>
__device__ __forceinline__ bool find_expert(const Args &a, int want, int &e, int &lo, int &hi) {
  e = want, lo = 0, hi = a.R;
  if (a.start) {
    if (a.E > a.R) {
      const int lane = threadIdx.x & (kWave - 1);
      int found = -1;
      for (int e0 = 0; e0 < a.E && found < 0; e0 += kWave) {
        const int f = e0 + lane;
        const bool some = f < a.E && row_bound(a.start, f + 1, a.R) > row_bound(a.start, f, a.R);
        unsigned long long m = __ballot(some);
        const int n = __popcll(m);
        if (want < n) {
          for (; want > 0; --want) m &= m - 1;
          found = e0 + __ffsll((long long)m) - 1;
        } else {
          want -= n;
        }
      }
      if (found < 0) return false;
      e = found;
    }
    lo = row_bound(a.start, e, a.R), hi = row_bound(a.start, e + 1, a.R);
  }
  return lo < hi;
}

struct RowTile {
  int e, m0, hi, nt;  // e < 0: nothing to do
};

// Item of workgroup `bid`: the row tiles (BM rows of one expert) times the
// ncols column tiles, expert by expert, inside an expert column outer and
// row tile inner, cut into eight equal contiguous shares, one per XCD
// (workgroup b runs on XCD b % 8): workgroups that share a weight tile then
// sit on one XCD at about the same time.  Every wave looks its item up for
// itself: a lane counts the tiles of ceil(E / 64) experts, a scan over the
// lanes finds the expert.
template <typename Args>
__device__ __forceinline__ RowTile find_tile(const Args &a, int BM, int ncols, int bid) {
  constexpr int kXcd = 8;
  const int lane = threadIdx.x & (kWave - 1);
  const int per_lane = (a.E + kWave - 1) / kWave, e0 = lane * per_lane;
  int sum = 0;
  for (int i = 0; i < per_lane && e0 + i < a.E; ++i) {
    const int lo = a.start ? row_bound(a.start, e0 + i, a.R) : 0;
    const int hi = a.start ? row_bound(a.start, e0 + i + 1, a.R) : a.R;
    sum += hi > lo ? (hi - lo + BM - 1) / BM : 0;
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int u = __shfl_up(incl, d);
    if (lane >= d) incl += u;
  }
  const int total = __builtin_amdgcn_readlane(incl, kWave - 1);
  // (start[] that does not rise could ask for more than the grid holds)
  const int n = total * ncols;
  const int per = (n + kXcd - 1) / kXcd;
  const int x = bid % kXcd, j = bid / kXcd, L = x * per + j;
  if (j >= per || L >= n) return {-1, 0, 0, 0};
  const int tile = L / ncols;
  const int src = __ffsll((long long)__ballot(tile < incl)) - 1;
  int base = incl - sum, fe = 0, flo = 0, fhi = 0, fbase = 0, fnb = 1;
  for (int i = 0; i < per_lane && e0 + i < a.E; ++i) {
    const int lo = a.start ? row_bound(a.start, e0 + i, a.R) : 0;
    const int hi = a.start ? row_bound(a.start, e0 + i + 1, a.R) : a.R;
    const int nb = hi > lo ? (hi - lo + BM - 1) / BM : 0;
    if (tile >= base && tile < base + nb) fe = e0 + i, flo = lo, fhi = hi, fbase = base, fnb = nb;
    base += nb;
  }
  const int e = __builtin_amdgcn_readlane(fe, src), lo = __builtin_amdgcn_readlane(flo, src);
  const int hi = __builtin_amdgcn_readlane(fhi, src), before = __builtin_amdgcn_readlane(fbase, src);
  const int nb = __builtin_amdgcn_readlane(fnb, src);
  const int r = L - before * ncols;
  return {e, lo + r % nb * BM, hi, r / nb};
}

}  // namespace moelora
