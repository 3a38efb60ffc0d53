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
// Everything is computed in float32, sums over tokens in float32 by lane and in
// 64 bits over the workgroups, always in the same order.
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

// e^x for x <= 0 (below 2^-126 zero): 2^y with the rounding of y = x log2(e)
// made good, within 2^-22 of the value.
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kLog2e = 0x1.715476p0f, kRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;  // log2(e) in two
  x = fmaxf(x, -200.f);
  const float y = x * kLog2e;
  const float rest = fmaf(x, kRest, fmaf(x, kLog2e, -y));
  const float p = __builtin_amdgcn_exp2f(y);
  return fmaf(p, rest * kLn2, p);
}
// e^(v - top); an infinite top shares the weight among its equals.
__device__ __forceinline__ float exp_below(float v, float top) { return v == top ? 1.f : exp_neg(v - top); }

// A group's share of one token.
template <int L, int S, typename DT> struct Row {
  static constexpr int C = S * sizeof(DT) < 16 ? S : 16 / (int)sizeof(DT);
  float v[S];  // logits of experts expert(i), kNone where not available

  __device__ __forceinline__ static int expert(int l, int i) { return (i / C * L + l) * C + i % C; }

  __device__ __forceinline__ void load(const DT *row, int E, int l, bool live) {
    typedef uint32_t words __attribute__((ext_vector_type(C * sizeof(DT) / 4)));
    typedef words mem __attribute__((aligned(2)));
    struct Chunk {
      DT e[C];
    };
#pragma unroll
    for (int c = 0; c < S / C; ++c) {
      const int e0 = expert(l, c * C);
      Chunk f;
      if (live && e0 + C <= E) {
        f = __builtin_bit_cast(Chunk, (words) * reinterpret_cast<const mem *>(row + e0));
      } else {
#pragma unroll
        for (int i = 0; i < C; ++i) f.e[i] = live && e0 + i < E ? row[e0 + i] : DT(0);
      }
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float x = Elem<DT>::to_f32(f.e[i]);
        v[c * C + i] = live && e0 + i < E && x > kNone ? x : kNone;  // (NaN is not above it)
      }
    }
  }
  __device__ __forceinline__ float max() const {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < S; ++i) m = fmaxf(m, v[i]);
    return group_max<L>(m);
  }
  // v becomes e^(v - top), 0 where not available; returns their sum.
  __device__ __forceinline__ float exponentials(float top) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      v[i] = v[i] == kNone ? 0.f : exp_below(v[i], top);
      z += v[i];
    }
    return group_sum<L>(z);
  }
};

__device__ __forceinline__ bool token_live(const uint8_t *mask, int t) { return !mask || mask[t] != 0; }

template <int L, int S, bool ALL, typename DT>
__global__ __launch_bounds__(kThreads) void k_route(RouterArgs a, int *__restrict__ ids, float *__restrict__ w) {
  constexpr int G = kThreads / L;
  __shared__ int pick[G][kMaxK + 1];
  __shared__ float part[G][kMaxK + 1];
  const int l = threadIdx.x % L, g = threadIdx.x / L;
  const int t = blockIdx.x * G + g;
  if (t >= a.T) return;  // (whole groups; nothing below crosses groups)
  Row<L, S, DT> r;
  r.load(static_cast<const DT *>(a.logits) + (size_t)t * a.E, a.E, l, token_live(a.mask, t));
  const float top = r.max();
  float z = 0.f;
  if constexpr (ALL) {
    Row<L, S, DT> q = r;
    z = q.exponentials(top);
  }
  float m = top;
  for (int j = 0; j < a.k; ++j) {
    if (j) m = r.max();
    int e = 0x7fffffff;
#pragma unroll
    for (int i = S - 1; i >= 0; --i) e = r.v[i] == m ? Row<L, S, DT>::expert(l, i) : e;
    e = group_min<L>(e);
#pragma unroll
    for (int i = 0; i < S; ++i) r.v[i] = Row<L, S, DT>::expert(l, i) == e ? kNone : r.v[i];
    const bool some = m > kNone;
    const float ex = some ? exp_below(m, top) : 0.f;
    if constexpr (!ALL) z += ex;
    if (l == 0) {
      pick[g][j] = some ? e : -1;
      part[g][j] = ex;
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  for (int j = l; j < a.k; j += L) {
    ids[(size_t)t * a.k + j] = pick[g][j];
    w[(size_t)t * a.k + j] = z > 0.f ? part[g][j] / z : 0.f;
  }
}

// Sums over the tokens of a chunk (workgroup b takes every gridDim.x-th set of
// G): the probabilities by expert, the picks by expert, the tokens and lse^2.
constexpr int kSumThreads = 512, kSumWaves = kSumThreads / kWave;

struct Totals {  // over the whole batch, in LDS
  double loss[kSumWaves];
};

// Counts, sums and losses from the chunks' sums: one workgroup.
__device__ void finish_losses(const RouterArgs &a, const BalanceOut &o, const float *sums, const int *counts,
                              const float *lse2, const int *live, int chunks, Totals &tot) {
  const int tid = threadIdx.x;
  double loss = 0.0;
  for (int e = tid; e < a.E; e += kSumThreads) {
    double s = 0.0;
    int c = 0;
    for (int b = 0; b < chunks; ++b) {
      s += sums[(size_t)b * a.E + e];
      c += counts[(size_t)b * a.E + e];
    }
    o.prob_sum[e] = (float)s;
    o.counts[e] = c;
    loss += s * c;
  }
#pragma unroll
  for (int d = kWave / 2; d >= 1; d >>= 1) loss += __shfl_xor(loss, d);
  if (tid % kWave == 0) tot.loss[tid / kWave] = loss;
  __syncthreads();
  if (tid == 0) {
    double s = 0.0, z = 0.0;
    int n = 0;
    for (int i = 0; i < kSumWaves; ++i) s += tot.loss[i];
    for (int b = 0; b < chunks; ++b) {
      z += lse2[b];
      n += live[b];
    }
    o.counts[a.E] = n;
    const double nd = n > 0 ? n : 1;
    o.loss[0] = (float)(s * a.E / (a.k * nd * nd));
    o.loss[1] = (float)(z / nd);
  }
}

template <int L, int S, typename DT>
__global__ __launch_bounds__(kSumThreads) void k_balance(RouterArgs a, const int *__restrict__ ids, BalanceOut o,
                                                         float *__restrict__ sums, int *__restrict__ counts,
                                                         float *__restrict__ lse2, int *__restrict__ lives) {
  constexpr int G = kSumThreads / L;
  __shared__ int hist[L * S];
  __shared__ float psum[kSumWaves][L * S];
  __shared__ float zs[kSumWaves];
  __shared__ int ns[kSumWaves];
  __shared__ Totals tot;
  __shared__ float one_z;
  __shared__ int one_n;
  const int tid = threadIdx.x, l = tid % L, g = tid / L, lane = tid % kWave, wave = tid / kWave;
  for (int e = tid; e < a.E; e += kSumThreads) hist[e] = 0;
  __syncthreads();
  float acc[S];
#pragma unroll
  for (int i = 0; i < S; ++i) acc[i] = 0.f;
  float z = 0.f;
  int n = 0;
  for (int t = blockIdx.x * G + g; t < a.T; t += gridDim.x * G) {
    Row<L, S, DT> r;
    r.load(static_cast<const DT *>(a.logits) + (size_t)t * a.E, a.E, l, token_live(a.mask, t));
    const float top = r.max();
    if (top == kNone) continue;  // (the same for the whole group)
    const float sum = r.exponentials(top), inv = 1.f / sum, lse = top + logf(sum);
#pragma unroll
    for (int i = 0; i < S; ++i) acc[i] += r.v[i] * inv;
    z += lse * lse;
    ++n;
    for (int j = l; j < a.k; j += L) {
      const int e = ids[(size_t)t * a.k + j];
      if ((unsigned)e < (unsigned)a.E) atomicAdd(&hist[e], 1);
    }
  }
  // the wave's groups, then the waves
#pragma unroll
  for (int d = L; d < kWave; d <<= 1) {
#pragma unroll
    for (int i = 0; i < S; ++i) acc[i] += __shfl_xor(acc[i], d);
    z += __shfl_xor(z, d);
    n += __shfl_xor(n, d);
  }
  if (lane < L) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int e = Row<L, S, DT>::expert(l, i);
      if (e < a.E) psum[wave][e] = acc[i];
    }
  }
  if (lane == 0) zs[wave] = z, ns[wave] = n;
  __syncthreads();
  const bool one = gridDim.x == 1;
  float *const out = sums + (size_t)blockIdx.x * a.E;
  for (int e = tid; e < a.E; e += kSumThreads) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kSumWaves; ++i) s += psum[i][e];
    if (one) {
      psum[0][e] = s;  // (each thread its own experts)
    } else {
      out[e] = s;
      counts[(size_t)blockIdx.x * a.E + e] = hist[e];
    }
  }
  if (tid == 0) {
    float s = 0.f;
    int c = 0;
    for (int i = 0; i < kSumWaves; ++i) s += zs[i], c += ns[i];
    if (one) one_z = s, one_n = c;
    else lse2[blockIdx.x] = s, lives[blockIdx.x] = c;
  }
  if (one) {
    __syncthreads();
    finish_losses(a, o, &psum[0][0], hist, &one_z, &one_n, 1, tot);
  }
}

__global__ __launch_bounds__(kSumThreads) void k_balance_finish(RouterArgs a, BalanceOut o, const float *sums,
                                                                const int *counts, const float *lse2,
                                                                const int *lives, int chunks) {
  __shared__ Totals tot;
  finish_losses(a, o, sums, counts, lse2, lives, chunks, tot);
}

template <int L, int S, bool ALL, typename DT>
__global__ __launch_bounds__(kThreads) void k_route_backward(RouterArgs a, RouteGradArgs q) {
  constexpr int G = kThreads / L;
  typedef Row<L, S, DT> R;
  const int l = threadIdx.x % L, g = threadIdx.x / L;
  float c[S], ca = 0.f, cz = 0.f;
#pragma unroll
  for (int i = 0; i < S; ++i) c[i] = 0.f;
  if (q.counts) {
    const int n = q.counts[a.E];
    const int mean = (int)((long long)a.k * n / a.E);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int e = R::expert(l, i);
      c[i] = e < a.E ? (float)(int)((unsigned)q.counts[e] - (unsigned)mean) : 0.f;
    }
    if (n > 0) {
      ca = q.dloss[0] * (float)a.E / ((float)a.k * (float)n) / (float)n;
      cz = q.dloss[1] * 2.f / (float)n;
    }
  }
  for (int t = blockIdx.x * G + g; t < a.T; t += gridDim.x * G) {
    R r;
    r.load(static_cast<const DT *>(a.logits) + (size_t)t * a.E, a.E, l, token_live(a.mask, t));
    float d[S];
    const int *id = q.ids + (size_t)t * a.k;
    const float *w = q.w + (size_t)t * a.k, *dw = q.dw + (size_t)t * a.k;  // (read where dw is given)
    float dot = 0.f;
    if (q.dw) {
      for (int j = l; j < a.k; j += L)
        if ((unsigned)id[j] < (unsigned)a.E) dot += w[j] * dw[j];
      dot = group_sum<L>(dot);
    }
    bool off[S];
#pragma unroll
    for (int i = 0; i < S; ++i) off[i] = r.v[i] == kNone;
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
      const float lse = top + logf(sum);
#pragma unroll
      for (int i = 0; i < S; ++i)
        d[i] = r.v[i] > 0.f ? r.v[i] * (fmaf(ca, c[i] - cp, cz * lse) - (ALL ? dot : 0.f)) : 0.f;
    } else {
#pragma unroll
      for (int i = 0; i < S; ++i) d[i] = 0.f;
    }
    if (q.dw) {
      for (int j = 0; j < a.k; ++j) {
        const int e = id[j];
        const float v = w[j] * (ALL ? dw[j] : dw[j] - dot);
#pragma unroll
        for (int i = 0; i < S; ++i) d[i] += R::expert(l, i) == e ? v : 0.f;
      }
    }
    DT *row = static_cast<DT *>(q.dlogits) + (size_t)t * a.E;
    constexpr int C = R::C;
#pragma unroll
    for (int ch = 0; ch < S / C; ++ch) {
      typedef uint32_t words __attribute__((ext_vector_type(C * sizeof(DT) / 4)));
      typedef words mem __attribute__((aligned(2)));
      struct {
        DT e[C];
      } f;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float v = off[ch * C + i] ? 0.f : d[ch * C + i];
        if constexpr (sizeof(DT) == 2) f.e[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
        else f.e[i] = v;
      }
      const int e0 = R::expert(l, ch * C);
      if (e0 + C <= a.E) {
        *reinterpret_cast<mem *>(row + e0) = __builtin_bit_cast(words, f);
      } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
          if (e0 + i < a.E) row[e0 + i] = f.e[i];
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

template <bool ALL, typename DT> struct BackwardLaunch {
  const RouterArgs &a;
  const RouteGradArgs &q;
  hipStream_t st;
  template <int L, int S> hipError_t operator()() {
    constexpr int G = kThreads / L;
    const int wgs = (a.T + G - 1) / G;
    return launch_kernel(k_route_backward<L, S, ALL, DT>, dim3(wgs < 4096 ? wgs : 4096), dim3(kThreads), 0, st, a,
                         q);
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
    float *sums = static_cast<float *>(ws);
    int *counts = reinterpret_cast<int *>(sums + (size_t)chunks * a.E);
    float *lse2 = reinterpret_cast<float *>(counts + (size_t)chunks * a.E);
    int *lives = reinterpret_cast<int *>(lse2 + chunks);
    hipError_t e = launch_kernel(k_balance<L, S, DT>, dim3(chunks), dim3(kSumThreads), 0, st, a, ids, o, sums, counts,
                                 lse2, lives);
    if (e != hipSuccess || (chunks == 1 && !tl_resolve_only)) return e;
    return launch_kernel(k_balance_finish, dim3(1), dim3(kSumThreads), 0, st, a, o, (const float *)sums,
                         (const int *)counts, (const float *)lse2, (const int *)lives, chunks);
  }
};

}  // namespace

int balance_chunks(int T, int E) {
  // one workgroup, and one launch, up to 32768 logits; then 32 tokens and more a chunk
  if ((long long)T * E <= 32768) return 1;
  const int c = (T + 31) / 32;
  return c < kBalanceChunks ? c : kBalanceChunks;
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
