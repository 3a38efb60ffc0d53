// The router by itself: picks and weights from logits, the balance and
// logsumexp losses over a batch, and the gradient of all three.
//
// With l[t][e] the logits, an expert is available to a token whose mask byte
// is set if its logit is above -inf and not NaN.  p = softmax over the
// available experts, lse its logarithm of the sum, n the tokens with any:
//     picks    the k largest available logits, ties to the lower expert
//     weights  softmax over the picks, or their p
//     losses   E / (k n^2) sum_e c[e] S[e] with c the picks and S the summed p
//              of each expert, and sum_t lse^2 / n
//     gradient dl_i = [i = id_j] w_j g_j - w_j or p_i times sum w g
//                     + p_i (a (c_i - sum_e c_e p_e) + z lse)
// A balanced router has counts near their mean, so c_i - sum c p would cancel:
// since sum p = 1 any whole number may be taken off all counts first, which is
// exact, and the mean is.
//
// A token belongs to L lanes side by side that hold its E logits in registers,
// S each, in chunks of C neighbours (one 16-byte load where that is as many), so
// a wave works on 64 / L tokens at once and a maximum or a sum over the experts
// is S steps in registers and log2 L across lanes, by DPP up to 16 lanes.
// Everything is computed in float32, sums over tokens in float32 inside a workgroup (its
// lanes, then its waves) and in 64 bits over the workgroups, always in the same order.
//
// Few tokens: a launch of 2 to 8 us, bound by its latency.  Many: the bytes could pass in
// half the time or less.  The picks are bound by the issue of the passes over S and of the
// steps across lanes (65536 x 256 bf16, 8 picks of the full softmax: 17.2 us of 7.5 for the bytes,
// the vector units busy 71 %), the losses and the gradient by the latency of a token's chain,
// maximum, exponentials, sum and what needs the sum, at four waves a SIMD (65521 x 128 float32
// 12 us, vector units busy 25 %; the gradient of 65521 x 256 bf16 27 us, 42 %).
#include "common.h"
#include "kernels.h"
#include "ops.h"

namespace moelora {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxK = 32;
constexpr float kNone = -__builtin_inff();  // an expert that cannot be picked (any more)

// DPP controls: quad permutations, half-row and row mirrors.
constexpr int kSwap1 = 0xb1, kSwap2 = 0x4e, kHalfMirror = 0x141, kMirror = 0x140;
template <int CTRL, typename T>
__device__ __forceinline__ T dpp(T v) {
  return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// v reduced over the group's L lanes, in every lane.  Each step joins two halves
// that hold one value each, so every lane adds the same numbers.
template <int L, typename T, typename F>
__device__ __forceinline__ T over_group(T v, F f) {
  v = f(v, dpp<kSwap1>(v));
  v = f(v, dpp<kSwap2>(v));
  if constexpr (L >= 8) v = f(v, dpp<kHalfMirror>(v));
  if constexpr (L >= 16) v = f(v, dpp<kMirror>(v));
  if constexpr (L >= 32) v = f(v, __shfl_xor(v, 16));
  if constexpr (L >= 64) v = f(v, __shfl_xor(v, 32));
  return v;
}
template <int L> __device__ __forceinline__ float group_max(float v) {
  return over_group<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L> __device__ __forceinline__ int group_min(int v) {
  return over_group<L>(v, [](int a, int b) { return min(a, b); });
}
template <int L> __device__ __forceinline__ float group_sum(float v) {
  return over_group<L>(v, [](float a, float b) { return a + b; });
}

// e^x for x <= 0 (below 2^-126, and of NaN, zero): 2^y with the rounding of y =
// x log2(e) made good, within 2^-22 of the value.
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kLog2e = 0x1.715476p0f, kRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;  // log2(e) in two
  x = fmaxf(x, -200.f);
  const float y = x * kLog2e;
  const float rest = fmaf(x, kRest, fmaf(x, kLog2e, -y));
  const float p = __builtin_amdgcn_exp2f(y);
  return fmaf(p, rest * kLn2, p);
}
// A group's share of one token.
template <int L, int S, typename DT> struct Row {
  static constexpr int C = S * sizeof(DT) < 16 ? S : 16 / (int)sizeof(DT);
  typedef uint32_t words __attribute__((ext_vector_type(C * sizeof(DT) / 4)));
  typedef words mem __attribute__((aligned(2)));
  struct Chunk {
    DT e[C];
  };
  float v[S];  // logits of experts expert(l, i), kNone where not available

  __device__ __forceinline__ static int expert(int l, int i) { return (i / C * L + l) * C + i % C; }

  // As they are stored, so that a token's can be on their way while another's are worked on.
  struct Raw {
    words w[S / C];
  };
  __device__ __forceinline__ static Raw load(const DT *row, int E, int l) {
    Raw r;
#pragma unroll
    for (int c = 0; c < S / C; ++c) {
      const int e0 = expert(l, c * C);
      if (e0 + C <= E) {
        r.w[c] = *reinterpret_cast<const mem *>(row + e0);
      } else {
        Chunk f;
#pragma unroll
        for (int i = 0; i < C; ++i) f.e[i] = e0 + i < E ? row[e0 + i] : DT(0);
        r.w[c] = __builtin_bit_cast(words, f);
      }
    }
    return r;
  }
  __device__ __forceinline__ void take(const Raw &r, int E, int l, bool live) {
#pragma unroll
    for (int c = 0; c < S / C; ++c) {
      const Chunk f = __builtin_bit_cast(Chunk, r.w[c]);
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float x = Elem<DT>::to_f32(f.e[i]);
        v[c * C + i] = x > kNone ? x : kNone;  // (NaN is not above it)
      }
    }
    if (E < L * S) {
#pragma unroll
      for (int i = 0; i < S; ++i) v[i] = expert(l, i) < E ? v[i] : kNone;
    }
    if (!__all(live)) {
#pragma unroll
      for (int i = 0; i < S; ++i) v[i] = live ? v[i] : kNone;
    }
  }
  __device__ __forceinline__ float max() const {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < S; ++i) m = fmaxf(m, v[i]);
    return group_max<L>(m);
  }
  // v becomes e^(v - top), 0 where not available (also where none is: NaN counts
  // as -200); of infinite logits each 1.  Returns their sum.
  __device__ __forceinline__ float exponentials(float top) {
    const bool inf = top == -kNone;
    if (__builtin_expect(__any(inf), 0)) {
#pragma unroll
      for (int i = 0; i < S; ++i) v[i] = inf ? (v[i] == top ? 1.f : 0.f) : exp_neg(v[i] - top);
    } else {
#pragma unroll
      for (int i = 0; i < S; ++i) v[i] = exp_neg(v[i] - top);
    }
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < S; ++i) z += v[i];
    return group_sum<L>(z);
  }
};

__device__ __forceinline__ bool token_live(const uint8_t *mask, int t) { return !mask || mask[t] != 0; }

// Picks by keys: the upper bits of a number that rises with the logit, and below
// them the expert's index counted down, so the largest key is the largest logit of
// the lowest index, and all keys differ.  The largest key below w is w plus the
// largest (key - w), modulo 2^32: one subtraction and half a three-way maximum a
// logit and pick, and nothing to strike out.  bf16 logits fit beside the
// index; of a float32 the index takes the last log2(L S) bits, and where two of a
// token's k + 1 largest keys agree in what is left, its wave picks once more by
// whole logits.  (65536 tokens, 8 of 256 experts, full softmax, bf16 17 us; by a maximum
// and its first index, struck out, 31.)
constexpr uint32_t kSign = 0x80000000u;
__device__ __forceinline__ uint32_t rising(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // (-0 becomes 0, which it equals)
  return u ^ ((uint32_t)((int)u >> 31) | kSign);
}
constexpr uint32_t kNoKey = 0x007fffffu;  // keys of -inf end here
// The bf16 value in the upper half of a key.
__device__ __forceinline__ float falling(uint32_t key) {
  return __uint_as_float((key & kSign ? key ^ kSign : ~key) & 0xffff0000u);
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <int L, int S, bool ALL, typename DT>
__global__ __launch_bounds__(kThreads) void k_route(RouterArgs a, int *__restrict__ ids, float *__restrict__ w) {
  constexpr int G = kThreads / L;
  constexpr bool EXACT = sizeof(DT) == 2;
  constexpr uint32_t INDEX = EXACT ? 0xffffu : L * S - 1;
  typedef Row<L, S, DT> R;
  __shared__ uint32_t pick[G][kMaxK + 1];
  const int l = threadIdx.x % L, g = threadIdx.x / L;
  const int t = blockIdx.x * G + g;
  if (t >= a.T) return;  // (whole groups; nothing below crosses groups)
  const DT *const row = static_cast<const DT *>(a.logits) + (size_t)t * a.E;
  R r;
  r.take(R::load(row, a.E, l), a.E, l, token_live(a.mask, t));
  uint32_t key[S];
#pragma unroll
  for (int i = 0; i < S; ++i) key[i] = (rising(r.v[i]) & ~INDEX) | (INDEX - R::expert(l, i));
  uint32_t last = 0;  // keys below 0, modulo 2^32: all of them
  bool close = false;
  for (int j = 0; j < a.k + (EXACT ? 0 : 1); ++j) {
    uint32_t d = 0;
#pragma unroll
    for (int i = 0; i < S; ++i) d = umax(d, key[i] - last);
    const uint32_t now = last + over_group<L>(d, umax);
    if (!EXACT) close |= j > 0 && now > kNoKey && !((now ^ last) & ~INDEX);
    last = now;
    if (l == 0 && j < a.k) pick[g][j] = now;
  }
  if (!EXACT && __any(close)) {
    R q = r;
    for (int j = 0; j < a.k; ++j) {
      const float m = q.max();
      int e = 0x7fffffff;
#pragma unroll
      for (int i = S - 1; i >= 0; --i) e = q.v[i] == m ? R::expert(l, i) : e;
      e = group_min<L>(e);
#pragma unroll
      for (int i = 0; i < S; ++i) q.v[i] = R::expert(l, i) == e ? kNone : q.v[i];
      if (l == 0) pick[g][j] = m > kNone ? ~INDEX | (INDEX - e) : 0u;
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  // pick j belongs to lane j % L from here on
  constexpr int PER = (kMaxK + L - 1) / L;
  int id[PER];
  float x[PER], top = kNone, z = 0.f;
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    if (u * L >= a.k) break;
    const int j = u * L + l;
    const uint32_t k = pick[g][min(j, a.k - 1)];
    id[u] = j < a.k && k > kNoKey ? (int)(INDEX - (k & INDEX)) : -1;
    x[u] = EXACT ? falling(k) : Elem<DT>::to_f32(row[max(id[u], 0)]);
    x[u] = id[u] >= 0 ? x[u] : kNone;
    top = fmaxf(top, x[u]);
  }
  top = group_max<L>(top);  // (the first pick's)
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    if (u * L >= a.k) break;
    x[u] = top == -kNone ? (x[u] == top ? 1.f : 0.f) : exp_neg(x[u] - top);
    z += x[u];
  }
  if constexpr (ALL) z = r.exponentials(top);
  else z = group_sum<L>(z);
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int j = u * L + l;
    if (u * L >= a.k) break;
    if (j < a.k) {
      ids[(size_t)t * a.k + j] = id[u];
      w[(size_t)t * a.k + j] = z > 0.f ? x[u] / z : 0.f;
    }
  }
}

// Sums over the tokens of a chunk (workgroup b takes every gridDim.x-th set of
// G): the probabilities by expert, the picks by expert, the tokens and lse^2, into
// the workspace; a batch of one chunk goes on to the losses by itself.
constexpr int kSumThreads = 1024, kSumWaves = kSumThreads / kWave, kRows = kSumWaves / 2;

struct ChunkSums {   // of all chunks
  float *prob;       // [chunks][E]
  int *picks;        // [chunks][E]
  float *lse2;       // [chunks]
  int *tokens;       // [chunks]
  double *loss;      // [workgroups of the second launch] their experts' counts x prob_sum
  unsigned *done;    // how many of those have finished
  int chunks;
};

// From sum_e counts prob_sum, sum lse^2 and the number of tokens.
__device__ __forceinline__ void write_losses(const RouterArgs &a, const BalanceOut &o, double s, double z, int n) {
  const double nd = n > 0 ? n : 1;
  o.counts[a.E] = n;
  o.loss[0] = (float)(s * a.E / (a.k * nd * nd));
  o.loss[1] = (float)(z / nd);
}

template <int L, int S, typename DT>
__global__ __launch_bounds__(kSumThreads) void k_balance(RouterArgs a, const int *__restrict__ ids, BalanceOut o,
                                                         ChunkSums c) {
  constexpr int G = kSumThreads / L;
  typedef Row<L, S, DT> R;
  __shared__ int hist[L * S];
  __shared__ float psum[kRows][L * S];
  __shared__ float zs[kSumWaves];
  __shared__ int ns[kSumWaves];
  __shared__ double part[kSumWaves];
  const int tid = threadIdx.x, l = tid % L, g = tid / L, lane = tid % kWave, wave = tid / kWave;
  if (blockIdx.x == 0 && tid == 0 && gridDim.x > 1) *c.done = 0;
  for (int e = tid; e < a.E; e += kSumThreads) hist[e] = 0;
  __syncthreads();
  float acc[S];
#pragma unroll
  for (int i = 0; i < S; ++i) acc[i] = 0.f;
  float z = 0.f;
  int n = 0;
  // a token's logits, mask and picks are loaded while the one before is worked on
  typename R::Raw raw;
  bool live = false;
  int id = -1;
  auto load = [&](int t) {
    const int at = min(t, a.T - 1);
    raw = R::load(static_cast<const DT *>(a.logits) + (size_t)at * a.E, a.E, l);
    live = token_live(a.mask, at);
    id = l < a.k ? ids[(size_t)at * a.k + l] : -1;
  };
  int t = blockIdx.x * G + g;
  if (t < a.T) load(t);
  for (; t < a.T; t += gridDim.x * G) {
    R r;
    r.take(raw, a.E, l, live);
    const int first = id;
    load(t + gridDim.x * G);
    const float top = r.max();
    if (top == kNone) continue;  // (the same for the whole group)
    const float sum = r.exponentials(top), inv = 1.f / sum, lse = top + logf(sum);
#pragma unroll
    for (int i = 0; i < S; ++i) acc[i] = fmaf(r.v[i], inv, acc[i]);
    z = fmaf(lse, lse, z);
    ++n;
    if ((unsigned)first < (unsigned)a.E) atomicAdd(&hist[first], 1);
    for (int j = l + L; j < a.k; j += L) {
      const int e = ids[(size_t)t * a.k + j];
      if ((unsigned)e < (unsigned)a.E) atomicAdd(&hist[e], 1);
    }
  }
  // the wave's groups, then the waves in two halves
#pragma unroll
  for (int d = L; d < kWave; d <<= 1) {
#pragma unroll
    for (int i = 0; i < S; ++i) acc[i] += __shfl_xor(acc[i], d);
    z += __shfl_xor(z, d);
    n += __shfl_xor(n, d);
  }
  if (lane == 0) zs[wave] = z, ns[wave] = n;
  if (wave >= kRows && lane < L) {
#pragma unroll
    for (int i = 0; i < S; ++i) psum[wave - kRows][R::expert(l, i)] = acc[i];
  }
  __syncthreads();
  if (wave < kRows && lane < L) {
#pragma unroll
    for (int i = 0; i < S; ++i) psum[wave][R::expert(l, i)] += acc[i];
  }
  __syncthreads();
  const bool one = gridDim.x == 1;
  float *const prob = one ? o.prob_sum : c.prob + (size_t)blockIdx.x * a.E;
  int *const picks = one ? o.counts : c.picks + (size_t)blockIdx.x * a.E;
  double loss = 0.0;
  for (int e = tid; e < a.E; e += kSumThreads) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) s += psum[i][e];
    prob[e] = s;
    picks[e] = hist[e];
    loss += (double)s * hist[e];
  }
  if (one) {
#pragma unroll
    for (int d = kWave / 2; d >= 1; d >>= 1) loss += __shfl_xor(loss, d);
    if (lane == 0) part[wave] = loss;
    __syncthreads();
  }
  if (tid > 0) return;
  float zt = 0.f;
  int nt = 0;
  for (int i = 0; i < kSumWaves; ++i) zt += zs[i], nt += ns[i];
  if (one) {
    loss = 0.0;
    for (int i = 0; i < kSumWaves; ++i) loss += part[i];
    write_losses(a, o, loss, zt, nt);
  } else {
    c.lse2[blockIdx.x] = zt;
    c.tokens[blockIdx.x] = nt;
  }
}

// Second launch: EX experts a workgroup, its threads spread over the chunks, added
// in 64 bits and in a fixed order.  Where there are several workgroups, the one that
// is last to finish adds up their shares of the loss (in the same order whichever
// it is).  16 experts a workgroup, or all of up to 128 where the chunks are few: one
// workgroup reads some 40 GB/s (6400 tokens of 32 experts 7.4 us, by several 8.4; 65521 of
// 128 16.5, by several 14.6).
constexpr int kFinishFew = 16, kFinishAll = 128;
template <int EX>
__global__ __launch_bounds__(kSumThreads) void k_balance_finish(RouterArgs a, BalanceOut o, ChunkSums c) {
  constexpr int PARTS = kSumThreads / EX, ROWS = EX < kWave ? kSumWaves : PARTS, BATCH = EX < kWave ? 4 : 8;
  __shared__ double prob[ROWS][EX];
  __shared__ int picks[ROWS][EX];
  const int tid = threadIdx.x, p = tid / EX, q = tid % EX;
  const int lane = tid % kWave, wave = tid / kWave;
  const int e0 = blockIdx.x * EX, e = min(e0 + q, a.E - 1);
  double s = 0.0;
  int n = 0;
  for (int b0 = p; b0 < c.chunks; b0 += BATCH * PARTS) {
    float f[BATCH];
    int m[BATCH];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const size_t at = (size_t)min(b0 + u * PARTS, c.chunks - 1) * a.E + e;
      f[u] = c.prob[at];
      m[u] = c.picks[at];
    }
#pragma unroll
    for (int u = 0; u < BATCH; ++u)
      if (b0 + u * PARTS < c.chunks) s += f[u], n += m[u];
  }
#pragma unroll
  for (int d = EX; d < kWave; d <<= 1) {
    s += __shfl_xor(s, d);
    n += __shfl_xor(n, d);
  }
  if (EX >= kWave || lane < EX) prob[EX < kWave ? wave : p][q] = s, picks[EX < kWave ? wave : p][q] = n;
  __syncthreads();
  if (wave > 0) return;
  double loss = 0.0;
  for (int i = lane; i < EX && e0 + i < a.E; i += kWave) {
    s = 0.0, n = 0;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) s += prob[r][i], n += picks[r][i];
    o.prob_sum[e0 + i] = (float)s, o.counts[e0 + i] = n;
    loss += (double)(float)s * n;
  }
#pragma unroll
  for (int d = kWave / 2; d >= 1; d >>= 1) loss += __shfl_xor(loss, d);
  if (gridDim.x > 1) {
    unsigned before = 0;
    if (lane == 0) {
      c.loss[blockIdx.x] = loss;
      before = __hip_atomic_fetch_add(c.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__builtin_amdgcn_readfirstlane(before) != gridDim.x - 1) return;
    static_assert(1024 / kFinishFew <= kWave, "a workgroup's share of the loss a lane");
    loss = lane < (int)gridDim.x ? c.loss[lane] : 0.0;
#pragma unroll
    for (int d = kWave / 2; d >= 1; d >>= 1) loss += __shfl_xor(loss, d);
  }
  double z = 0.0;
  n = 0;
  for (int b = lane; b < c.chunks; b += kWave) z += c.lse2[b], n += c.tokens[b];
#pragma unroll
  for (int d = kWave / 2; d >= 1; d >>= 1) {
    z += __shfl_xor(z, d);
    n += __shfl_xor(n, d);
  }
  if (lane == 0) write_losses(a, o, loss, z, n);
}

// The picks' terms come to the lanes that own their experts through a row in LDS
// for each group, zero but for the picks: lane j writes the j-th's value there, all
// lanes read theirs, lane j writes zero again.  Ids that a caller repeats would meet in one place:
// lane j writes j first and looks whether it stays; if any does not, the
// wave's tokens add theirs one after the other.  (65536 x 256 bf16, 8 picks of the full
// softmax, with the balance gradient: 27 us, 14.5 for the bytes; every lane comparing all
// picks with its experts 49.)
template <int L, int S, bool ALL, typename DT>
__global__ __launch_bounds__(kThreads) void k_route_backward(RouterArgs a, RouteGradArgs q) {
  constexpr int G = kThreads / L, PER = (kMaxK + L - 1) / L;
  typedef Row<L, S, DT> R;
  __shared__ float terms[G][L * S];
  const int l = threadIdx.x % L, g = threadIdx.x / L;
  float *const mine = terms[g];
#pragma unroll
  for (int i = 0; i < S; ++i) mine[R::expert(l, i)] = 0.f;
  // a token's logits, mask and picks are loaded while the one before is worked on;
  // pick j belongs to lane j % L
  struct Token {
    typename R::Raw raw;
    bool live;
    int id[PER];
    float w[PER], dw[PER];
  } next;
  auto load = [&](int t) {
    t = min(t, a.T - 1);
    next.raw = R::load(static_cast<const DT *>(a.logits) + (size_t)t * a.E, a.E, l);
    next.live = token_live(a.mask, t);
    if (q.dw) {
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        if (u * L >= a.k) break;
        const size_t at = (size_t)t * a.k + min(u * L + l, a.k - 1);
        next.id[u] = q.ids[at];
        next.w[u] = q.w[at], next.dw[u] = q.dw[at];
      }
    }
  };
  int t = blockIdx.x * G + g;
  load(t);
  float c[S], ca = 0.f, cz = 0.f;
#pragma unroll
  for (int i = 0; i < S; ++i) c[i] = 0.f;
  if (q.counts) {
    const int n = q.counts[a.E];
    const int mean = (int)((long long)a.k * n / a.E);
#pragma unroll
    for (int i = 0; i < S; ++i)
      c[i] = (float)(int)((unsigned)q.counts[min(R::expert(l, i), a.E)] - (unsigned)mean);  // (past E: of no use)
    if (n > 0) {
      ca = q.dloss[0] * (float)a.E / ((float)a.k * (float)n) / (float)n;
      cz = q.dloss[1] * 2.f / (float)n;
    }
  }
  for (; t < a.T; t += gridDim.x * G) {
    R r;
    r.take(next.raw, a.E, l, next.live);
    int id[PER];
    float v[PER], x[PER], dot = 0.f;
    if (q.dw) {
      float w[PER];
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        if (u * L >= a.k) break;
        const bool ok = u * L + l < a.k && (unsigned)next.id[u] < (unsigned)a.E;
        id[u] = ok && next.live ? next.id[u] : -1;
        w[u] = ok ? next.w[u] : 0.f, v[u] = ok ? next.dw[u] : 0.f;
        dot = fmaf(w[u], v[u], dot);
        // (an expert that is not available has no gradient, whoever picked it)
        x[u] = Elem<DT>::to_f32((static_cast<const DT *>(a.logits) + (size_t)t * a.E)[max(id[u], 0)]);
      }
      dot = group_sum<L>(dot);
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        if (u * L >= a.k) break;
        v[u] = w[u] * (ALL ? v[u] : v[u] - dot);
      }
    }
    load(t + gridDim.x * G);
    float d[S];
    if (ALL || q.counts) {
      const float top = r.max();
      const float sum = r.exponentials(top), inv = sum > 0.f ? 1.f / sum : 0.f;
      float cp = 0.f;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        r.v[i] *= inv;
        cp = fmaf(c[i], r.v[i], cp);
      }
      cp = group_sum<L>(cp);
      // (of infinite logits lse is infinite: nothing of it where its loss has no gradient)
      const float rest = (cz != 0.f ? cz * (top + logf(sum)) : 0.f) - (ALL ? dot : 0.f);
#pragma unroll
      for (int i = 0; i < S; ++i) d[i] = r.v[i] > 0.f ? r.v[i] * fmaf(ca, c[i] - cp, rest) : 0.f;
    } else {
#pragma unroll
      for (int i = 0; i < S; ++i) d[i] = 0.f;
    }
    if (q.dw) {
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        if (u * L >= a.k) break;
        id[u] = x[u] > kNone ? id[u] : -1;
      }
      const auto each = [&](auto f) {
#pragma unroll
        for (int u = 0; u < PER; ++u) {
          if (u * L >= a.k) break;
          if (id[u] >= 0) f(u);
        }
      };
      bool twice = false;
      each([&](int u) { mine[id[u]] = __int_as_float(u * L + l + 1); });
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      each([&](int u) { twice |= __float_as_int(mine[id[u]]) != u * L + l + 1; });
      if (__builtin_expect(__any(twice), 0)) {
        each([&](int u) { mine[id[u]] = 0.f; });
        for (int j = 0; j < a.k; ++j) {
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          each([&](int u) {
            if (u * L + l == j) mine[id[u]] += v[u];
          });
        }
      } else {
        each([&](int u) { mine[id[u]] = v[u]; });
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int i = 0; i < S; ++i) d[i] += mine[R::expert(l, i)];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      each([&](int u) { mine[id[u]] = 0.f; });
    }
    DT *const out = static_cast<DT *>(q.dlogits) + (size_t)t * a.E;
    constexpr int C = R::C;
#pragma unroll
    for (int ch = 0; ch < S / C; ++ch) {
      typename R::Chunk f;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float x = d[ch * C + i];
        if constexpr (sizeof(DT) == 2) f.e[i] = __builtin_bit_cast(uint16_t, (__bf16)x);
        else f.e[i] = x;
      }
      const int e0 = R::expert(l, ch * C);
      if (e0 + C <= a.E) {
        *reinterpret_cast<typename R::mem *>(out + e0) = __builtin_bit_cast(typename R::words, f);
      } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
          if (e0 + i < a.E) out[e0 + i] = f.e[i];
      }
    }
  }
}

// Lanes a token and logits a lane, by the number of experts.
template <typename F>
hipError_t by_experts(int E, F f) {
  if (E <= 16) return f.template operator()<4, 4>();
  if (E <= 32) return f.template operator()<8, 4>();
  if (E <= 64) return f.template operator()<8, 8>();
  if (E <= 128) return f.template operator()<16, 8>();
  if (E <= 256) return f.template operator()<16, 16>();
  if (E <= 512) return f.template operator()<32, 16>();
  return f.template operator()<64, 16>();
}

template <bool ALL, typename DT> struct RouteLaunch {
  const RouterArgs &a;
  int *ids;
  float *w;
  hipStream_t st;
  template <int L, int S> hipError_t operator()() {
    constexpr int G = kThreads / L;
    return launch_kernel(k_route<L, S, ALL, DT>, dim3((a.T + G - 1) / G), dim3(kThreads), 0, st, a, ids, w);
  }
};

// As many workgroups of the gradient as stay resident: each goes through several
// sets of tokens, loading one ahead.
constexpr int kBackwardWgs = 1024;
template <bool ALL, typename DT> struct BackwardLaunch {
  const RouterArgs &a;
  const RouteGradArgs &q;
  hipStream_t st;
  template <int L, int S> hipError_t operator()() {
    constexpr int G = kThreads / L;
    const int wgs = (a.T + G - 1) / G;
    return launch_kernel(k_route_backward<L, S, ALL, DT>, dim3(wgs < kBackwardWgs ? wgs : kBackwardWgs), dim3(kThreads), 0,
                         st, a, q);
  }
};

template <typename DT> struct BalanceLaunch {
  const RouterArgs &a;
  const int *ids;
  const BalanceOut &o;
  void *ws;
  int chunks;
  hipStream_t st;
  template <int L, int S> hipError_t operator()() {
    ChunkSums c;
    c.chunks = chunks;
    c.prob = static_cast<float *>(ws);
    c.picks = reinterpret_cast<int *>(c.prob + (size_t)chunks * a.E);
    c.lse2 = reinterpret_cast<float *>(c.picks + (size_t)chunks * a.E);
    c.tokens = reinterpret_cast<int *>(c.lse2 + chunks);
    c.done = reinterpret_cast<unsigned *>(c.tokens + chunks);
    // (chunks are even: the doubles are aligned)
    c.loss = reinterpret_cast<double *>(c.done + 2);
    hipError_t e = launch_kernel(k_balance<L, S, DT>, dim3(chunks), dim3(kSumThreads), 0, st, a, ids, o, c);
    if (e != hipSuccess || (chunks == 1 && !tl_resolve_only)) return e;
    if ((a.E <= kFinishAll && chunks * a.E <= 4096) || tl_resolve_only) {
      e = launch_kernel(k_balance_finish<kFinishAll>, dim3(1), dim3(kSumThreads), 0, st, a, o, c);
      if (e != hipSuccess || !tl_resolve_only) return e;
    }
    return launch_kernel(k_balance_finish<kFinishFew>, dim3((a.E + kFinishFew - 1) / kFinishFew), dim3(kSumThreads),
                         0, st, a, o, c);
  }
};

}  // namespace

// A workgroup's groups of lanes take a token each at a time.  Up to four rounds of
// that are left to one workgroup, and one launch (256 tokens of 128 experts 8.0 us, in
// two launches 7.7, but each costs the host 3).
struct GroupsOf {
  template <int L, int S> hipError_t operator()() {
    groups = kSumThreads / L;
    return hipSuccess;
  }
  int &groups;
};
int balance_chunks(int T, int E) {
  int groups = 1;
  (void)by_experts(E, GroupsOf{groups});
  if (T <= 4 * groups) return 1;
  const int c = (T + groups - 1) / groups;
  return c < kBalanceChunks ? (c + 1) / 2 * 2 : kBalanceChunks;
}

size_t balance_workspace(int T, int E) {
  const int c = balance_chunks(T, E);
  return c > 1 ? ((size_t)c * (2 * E + 2) + 2) * 4 + (E + kFinishFew - 1) / kFinishFew * sizeof(double) : 0;
}

hipError_t launch_route(const RouterArgs &a, bool all, bool bf16, int *ids, float *w, hipStream_t st) {
  if (all)
    return bf16 ? by_experts(a.E, RouteLaunch<true, uint16_t>{a, ids, w, st})
                : by_experts(a.E, RouteLaunch<true, float>{a, ids, w, st});
  return bf16 ? by_experts(a.E, RouteLaunch<false, uint16_t>{a, ids, w, st})
              : by_experts(a.E, RouteLaunch<false, float>{a, ids, w, st});
}

hipError_t launch_route_backward(const RouterArgs &a, const RouteGradArgs &q, bool all, bool bf16, hipStream_t st) {
  if (all)
    return bf16 ? by_experts(a.E, BackwardLaunch<true, uint16_t>{a, q, st})
                : by_experts(a.E, BackwardLaunch<true, float>{a, q, st});
  return bf16 ? by_experts(a.E, BackwardLaunch<false, uint16_t>{a, q, st})
              : by_experts(a.E, BackwardLaunch<false, float>{a, q, st});
}

hipError_t launch_balance(const RouterArgs &a, bool bf16, const int *ids, const BalanceOut &o, void *ws,
                          hipStream_t st) {
  const int chunks = balance_chunks(a.T, a.E);
  return bf16 ? by_experts(a.E, BalanceLaunch<uint16_t>{a, ids, o, ws, chunks, st})
              : by_experts(a.E, BalanceLaunch<float>{a, ids, o, ws, chunks, st});
}

}  // namespace moelora
