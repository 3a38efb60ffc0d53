// Token order: routed rows sorted by expert, tokens copied into that order,
// expert outputs added back per token, and the gradients of both.
//
// With p = t k + j the routed rows and e(p) their expert (rows with e(p)
// outside [0, E) dropped), the order is the stable one: pos(p) = #{q : e(q)
// < e(p)} + #{q < p : e(q) = e(p)}.  Then
//     dispatch            xs[pos(p)] = x[p / k]
//     its gradient        dx[t]      = sum_j dxs[pos(t, j)]
//     combine             out[t]     = sum_j w[t][j] ys[pos(t, j)]
//     its gradients       dys[pos(p)] = w[p] dout[p / k],
//                         dw[p]       = <dout[p / k], ys[pos(p)]>
// All sums run in float32 in ascending j (dw: a fixed tree), each result is
// rounded once, and nothing uses floating-point atomics, so results repeat
// bit for bit.  Everything but the order itself is bound by HBM: the copies
// read each token once and write each routed row once (and the reverse),
// 16 bytes a lane.  What is written or read once goes past the caches
// (non-temporal), which leaves them to the tokens and to the caller: the copy
// of 6400 x 2880 bf16 tokens for top-4 45.8 -> 35.6 us with its order (184 MB,
// 5.2 TB/s), their combine's gradients 75.7 -> 63.9 us (332 MB, 5.2 TB/s),
// combine 41.6 -> 39.5 us (33.7 with eight rows' loads together); nor does a
// consumer lose by it (dispatch, a library op, combine and back: 254 -> 247 us).
#include "common.h"
#include "kernels.h"
#include "ops.h"

namespace moelora {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxE = 1024;
// Up to this many routed rows one launch orders and copies: the workgroup of
// a row finds the row's place by counting (R comparisons), so that a decode
// step pays one launch.  us for 2880 and 80 bf16 columns on 32 experts, one
// launch against three: 64 rows 2.6 / 7.2, 2800 7.4 / 8.7 and 5.4 / 8.5, 4000 9.3 /
// 8.7 and 6.9 / 8.7, 6000 15.3 / 10.6.
constexpr int kFusedRows = 2800;
// Beyond that, up to this many, every workgroup of the order counts all the ids
// itself, which saves the launch that counts; its reads grow with R, those of
// the counts of all chunks with E.  us with 64 columns, two launches against
// three: 64 experts, 12000 rows 6.3 / 7.2, 24000 8.2 / 7.4; 256 experts, 32000 9.7 /
// 10.3, 64000 14.8 / 14.5; 1000 experts, 12000 7.7 / 13.1, 128000 29.9 / 40.7.
bool counts_itself(int R, int E) { return R <= 128 * (E > 128 ? E : 128); }

// What a lane moves at once, and how it lies in memory.  16-byte accesses need
// no more than 2-byte alignment here, so rows of any length are moved 16 bytes
// a lane: chunk c of a row starts at c steps of 16 bytes, the last one at the
// row's end less 16 (it may cover bytes of the one before once more, with the
// same values).  Rows shorter than 16 bytes go element by element.
template <int BYTES> struct Raw;
template <> struct Raw<16> {
  typedef u32x4_t type;
  typedef u32x4_t mem __attribute__((aligned(2)));
};
template <> struct Raw<4> {
  typedef uint32_t type;
  typedef uint32_t mem;
};
template <> struct Raw<2> {
  typedef uint16_t type;
  typedef uint16_t mem;
};
template <int BYTES>
__device__ __forceinline__ const typename Raw<BYTES>::mem *raw(const void *p) {
  return static_cast<const typename Raw<BYTES>::mem *>(p);
}
template <int BYTES>
__device__ __forceinline__ typename Raw<BYTES>::mem *raw(void *p) {
  return static_cast<typename Raw<BYTES>::mem *>(p);
}

__device__ __forceinline__ bool held(int e, int E) { return (unsigned)e < (unsigned)E; }

// One routed row per workgroup (0 .. R-1): its place, then its token's copy.
// Workgroup R writes expert_start and the sentinel tail of sorted_rows.
template <int BYTES>
__global__ __launch_bounds__(kThreads) void k_dispatch_fused(
    OrderShape s, int row_bytes, const char *__restrict__ x, const int *__restrict__ ids,
    int *__restrict__ expert_start, int *__restrict__ sorted_rows, int *__restrict__ row_pos,
    char *__restrict__ xs) {
  __shared__ int part[kWaves];
  __shared__ int hist[kMaxE];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int R = s.R, E = s.E;
  if ((int)blockIdx.x < R) {
    const int p = blockIdx.x;
    const int e = ids[p];
    if (!held(e, E)) {  // uniform: the whole workgroup leaves
      if (tid == 0) row_pos[p] = -1;
      return;
    }
    int n = 0;  // rows before p in the order, this wave's share (uniform)
    auto precedes = [&](int q, int f) { return q < R && held(f, E) && (f < e || (f == e && q < p)); };
    constexpr int kBatch = 8;  // ids on their way at once, where there are many
    int q0 = wave * kWave + lane;
    for (; R > 2 * kThreads && q0 - lane < R; q0 += kBatch * kThreads) {
      int f[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) f[u] = ids[min(q0 + u * kThreads, R - 1)];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) n += __popcll(__ballot(precedes(q0 + u * kThreads, f[u])));
    }
    for (; q0 - lane < R; q0 += kThreads)
      n += __popcll(__ballot(precedes(q0, q0 < R ? ids[q0] : -1)));
    if (lane == 0) part[wave] = n;
    __syncthreads();
    int pos = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) pos += part[w];
    if (tid == 0) {
      sorted_rows[pos] = p;
      row_pos[p] = pos;
    }
    if (xs) {
      const char *src = x + (size_t)(p / s.k) * row_bytes;
      char *dst = xs + (size_t)pos * row_bytes;
      for (int c = tid * BYTES; c < row_bytes; c += kThreads * BYTES) {
        const int o = min(c, row_bytes - BYTES);
        *raw<BYTES>(dst + o) = *raw<BYTES>(src + o);
      }
    }
    return;
  }
  for (int e = tid; e < E; e += kThreads) hist[e] = 0;
  __syncthreads();
  for (int q = tid; q < R; q += kThreads) {
    const int f = ids[q];
    if (held(f, E)) atomicAdd(&hist[f], 1);
  }
  __syncthreads();
  // wave 0: exclusive scan, each lane kMaxE / 64 experts in steps of 64
  if (wave == 0) {
    int base = 0;
    for (int e0 = 0; e0 < E; e0 += kWave) {
      const int e = e0 + lane;
      const int n = e < E ? hist[e] : 0;
      int v = n;
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) {
        const int u = __shfl_up(v, d);
        if (lane >= d) v += u;
      }
      if (e < E) expert_start[e] = base + v - n;
      base += __shfl(v, kWave - 1);
    }
    if (lane == 0) {
      expert_start[E] = base;
      part[0] = base;
    }
  }
  __syncthreads();
  for (int q = part[0] + tid; q < R; q += kThreads) sorted_rows[q] = R;
}

// Large batches, first launch: rows per expert of each chunk of C rows.
__global__ __launch_bounds__(kThreads) void k_order_count(int R, int E, int C,
                                                          const int *__restrict__ ids,
                                                          int *__restrict__ counts) {
  __shared__ int hist[kMaxE];
  const int tid = threadIdx.x;
  for (int e = tid; e < E; e += kThreads) hist[e] = 0;
  __syncthreads();
  const int lo = blockIdx.x * C, hi = min(R, lo + C);
  for (int q = lo + tid; q < hi; q += kThreads) {
    const int f = ids[q];
    if (held(f, E)) atomicAdd(&hist[f], 1);
  }
  __syncthreads();
  for (int e = tid; e < E; e += kThreads) counts[(size_t)blockIdx.x * E + e] = hist[e];
}

// Next launch: places of a chunk's rows, from the counts of all chunks or, with
// DIRECT, from the ids alone.  An expert's first place in the
// chunk is the experts before it plus the chunks before this one; the waves
// take a quarter of the chunk each, in order, 64 rows at a time: lanes with
// the same expert find each other by ballots over the bits of the id, and a
// lane's rank is the number of equal lanes below it.
template <bool DIRECT>
__global__ __launch_bounds__(kThreads) void k_order_place(
    int R, int E, int C, int nch, int id_bits, int e_shift, const int *__restrict__ ids,
    const int *__restrict__ counts, int *__restrict__ expert_start, int *__restrict__ sorted_rows,
    int *__restrict__ row_pos) {
  __shared__ int next[kWaves][kMaxE];
  __shared__ int before[kMaxE];
  __shared__ int part[2][DIRECT ? kMaxE : kThreads];
  __shared__ int wsum[kWaves];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int me = blockIdx.x;
  const int lo = me * C, hi = min(R, lo + C);
  const int quarter = (hi - lo + kWaves - 1) / kWaves;
  const int wlo = min(hi, lo + wave * quarter), whi = min(hi, wlo + quarter);
  for (int e = tid; e < kWaves * kMaxE; e += kThreads) (&next[0][0])[e] = 0;
  if constexpr (DIRECT)
    for (int e = tid; e < 2 * kMaxE; e += kThreads) (&part[0][0])[e] = 0;
  __syncthreads();
  constexpr int kBatch = 16;  // ids or counts on their way at once
  if constexpr (DIRECT) {  // part[0]: rows before the chunk, part[1]: the others
    for (int q0 = tid; q0 < R; q0 += kBatch * kThreads) {
      int f[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) f[u] = ids[min(q0 + u * kThreads, R - 1)];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int q = q0 + u * kThreads;
        if (q < R && held(f[u], E)) atomicAdd(&part[q >= lo][f[u]], 1);
      }
    }
  }
  for (int q = wlo + lane; q < whi; q += kWave) {
    const int f = ids[q];
    if (held(f, E)) atomicAdd(&next[wave][f], 1);
  }
  if constexpr (DIRECT) __syncthreads();
  // totals, and the chunks before this one: 2^e_shift experts at a time, the
  // chunks dealt over the kThreads >> e_shift threads of an expert
  const int per = 1 << e_shift, el = tid & (per - 1), gi = tid >> e_shift, G = kThreads >> e_shift;
  int kept = 0;
  for (int e0 = 0; e0 < E; e0 += per) {
    const int e = tid < per ? e0 + tid : E;  // the expert this thread scans for
    int total = 0, mine = 0;
    if constexpr (DIRECT) {
      if (e < E) {
        mine = part[0][e];
        total = mine + part[1][e];
      }
    } else if (e0 + el < E) {
      for (int c0 = gi; c0 < nch; c0 += kBatch * G) {
        int n[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          n[u] = counts[(size_t)min(c0 + u * G, nch - 1) * E + e0 + el];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int c = c0 + u * G;
          total += c < nch ? n[u] : 0;
          mine += c < me ? n[u] : 0;
        }
      }
    }
    if (!DIRECT && G > 1) {
      part[0][tid] = total;
      part[1][tid] = mine;
      __syncthreads();
      total = mine = 0;
      if (tid < per)
        for (int q = 0; q < G; ++q) {
          total += part[0][q * per + tid];
          mine += part[1][q * per + tid];
        }
    }
    int v = total;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int u = __shfl_up(v, d);
      if (lane >= d) v += u;
    }
    if (lane == kWave - 1) wsum[wave] = v;
    __syncthreads();
    int base = kept;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) base += wsum[w];
      kept += wsum[w];
    }
    if (e < E) {
      before[e] = base + v - total + mine;
      if (me == 0) expert_start[e] = base + v - total;
    }
    __syncthreads();
  }
  if (me == 0 && tid == 0) expert_start[E] = kept;
  for (int e = tid; e < E; e += kThreads) {
    int at = before[e];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const int n = next[w][e];
      next[w][e] = at;
      at += n;
    }
  }
  __syncthreads();
  for (int q0 = wlo; q0 < whi; q0 += kWave) {
    const int q = q0 + lane;
    const int f = q < whi ? ids[q] : -1;
    const bool ok = held(f, E);
    unsigned long long same = __ballot(ok);
    for (int b = 0; b < id_bits; ++b) {
      const unsigned long long on = __ballot(f >> b & 1);
      same &= (f >> b & 1) ? on : ~on;
    }
    if (ok) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      const int at = next[wave][f];  // read by every lane before the first writes it back
      const int pos = at + rank;
      sorted_rows[pos] = q;
      row_pos[q] = pos;
      if (rank == 0) next[wave][f] = at + __popcll(same);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    } else if (q < whi) {
      row_pos[q] = -1;
    }
  }
  // the sentinel tail, a share to each workgroup
  for (int q = kept + me * kThreads + tid; q < R; q += nch * kThreads) sorted_rows[q] = R;
}

// Threads a token and its tiles: one chunk a thread, `tpt` threads side by side.
struct RowGrid {
  int tpt_shift, tiles;
  dim3 grid;
};
RowGrid row_grid(int T, int chunks) {
  int best = 6;  // 64, 128 or 256 threads a token, whichever wastes fewest
  for (int sh = 7; sh <= 8; ++sh) {
    const int b = 1 << best, n = 1 << sh;
    if ((chunks + n - 1) / n * n <= (chunks + b - 1) / b * b) best = sh;
  }
  while (best > 0 && (1 << (best - 1)) >= chunks) --best;
  // (a launch holds fewer than 2^32 threads along x)
  while (((long long)T << best) > 0xffffff00ll - kThreads) --best;
  RowGrid g;
  g.tpt_shift = best;
  g.tiles = (chunks + (1 << best) - 1) >> best;
  const int per = kThreads >> best;
  g.grid = dim3((T + per - 1) / per, g.tiles);
  return g;
}

// A store past the caches where the wave, whose lanes store bytes [lo, hi) of
// `row` together, fills every line that this lane's bytes touch; through them
// for the lines at its ends, which other waves or rows complete (written past
// the caches a part at a time they cost HBM a pass each: rows of 2888 bf16,
// 6000 tokens for top-4, 43.9 -> 34.2 us, their combine's gradients 78.6 -> 59.3;
// of 2050, 12000 tokens, 71 -> 58; rows of whole lines are as they were).
template <int BYTES>
__device__ __forceinline__ void store_past(typename Raw<BYTES>::type v, char *row, int o, int lo, int hi) {
  constexpr uintptr_t kLine = 128;
  const uintptr_t a = reinterpret_cast<uintptr_t>(row);
  if (((a + o) & -kLine) >= a + lo && ((a + o + BYTES - 1) | (kLine - 1)) < a + hi) {
    __builtin_nontemporal_store(v, raw<BYTES>(row + o));
    asm volatile("");  // (or the compiler makes one plain store of the two)
  } else {
    *raw<BYTES>(row + o) = v;
  }
}

// xs[pos(t, j)] = x[t] for every j: a token is read once.
template <int BYTES>
__global__ __launch_bounds__(kThreads) void k_scatter(OrderShape s, int row_bytes, int tpt_shift,
                                                      const char *__restrict__ x,
                                                      const int *__restrict__ row_pos,
                                                      char *__restrict__ xs) {
  const int tpt = 1 << tpt_shift;
  const int t = blockIdx.x * (kThreads >> tpt_shift) + (threadIdx.x >> tpt_shift);
  const int c = blockIdx.y * tpt + (threadIdx.x & (tpt - 1));
  if (t >= s.T || c * BYTES >= row_bytes) return;
  const int o = min(c * BYTES, row_bytes - BYTES);
  const typename Raw<BYTES>::type v = *raw<BYTES>(x + (size_t)t * row_bytes + o);
  const int *pos = row_pos + (size_t)t * s.k;
  const int side = min(tpt, kWave);  // chunks of this row that the wave stores together
  const int lo = (c & -side) * BYTES, hi = min(lo + side * BYTES, row_bytes);
  for (int j = 0; j < s.k; ++j) {
    const int p = pos[j];
    if ((unsigned)p < (unsigned)s.R) store_past<BYTES>(v, xs + (size_t)p * row_bytes, o, lo, hi);
  }
}

// N elements of a row as float32.
template <typename DT, int N> struct Pack {
  DT v[N];
};
template <typename DT, int N>
__device__ __forceinline__ void unpack(typename Raw<sizeof(DT) * N>::type v, float *f) {
  const Pack<DT, N> a = __builtin_bit_cast(Pack<DT, N>, v);
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = Elem<DT>::to_f32(a.v[i]);
}
template <typename DT, int N>
__device__ __forceinline__ typename Raw<sizeof(DT) * N>::type pack(const float *f) {
  Pack<DT, N> a;
#pragma unroll
  for (int i = 0; i < N; ++i) a.v[i] = Elem<DT>::from_f32(f[i]);
  return __builtin_bit_cast(typename Raw<sizeof(DT) * N>::type, a);
}

// out[t] = sum_j w[t][j] ys[pos(t, j)], ascending j; the loads of eight rows
// are issued together.
template <typename DT, int N, bool WEIGHTED>
__global__ __launch_bounds__(kThreads) void k_combine_order(
    OrderShape s, int tpt_shift, const DT *__restrict__ ys, const int *__restrict__ row_pos,
    const float *__restrict__ w, DT *__restrict__ out) {
  constexpr int BYTES = sizeof(DT) * N;
  const int tpt = 1 << tpt_shift;
  const int t = blockIdx.x * (kThreads >> tpt_shift) + (threadIdx.x >> tpt_shift);
  const int c = blockIdx.y * tpt + (threadIdx.x & (tpt - 1));
  if (t >= s.T || c * N >= s.H) return;
  const int o = min(c * N, s.H - N);
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  const int k = s.k;
  const size_t r0 = (size_t)t * k;
  constexpr int kBatch = 8;
  for (int j0 = 0; j0 < k; j0 += kBatch) {
    typename Raw<BYTES>::type v[kBatch];
    float g[kBatch];
    int p[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      p[b] = j0 + b < k ? row_pos[r0 + j0 + b] : -1;
      g[b] = WEIGHTED && j0 + b < k ? w[r0 + j0 + b] : 1.f;
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if ((unsigned)p[b] < (unsigned)s.R)
        v[b] = __builtin_nontemporal_load(raw<BYTES>(ys + (size_t)p[b] * s.H + o));
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if ((unsigned)p[b] < (unsigned)s.R) {
        float f[N];
        unpack<DT, N>(v[b], f);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = WEIGHTED ? fmaf(g[b], f[i], acc[i]) : acc[i] + f[i];
      }
  }
  *raw<BYTES>(out + (size_t)t * s.H + o) = pack<DT, N>(acc);
}

// Up to this many routed rows a workgroup takes one, beyond it one per wave:
// few rows leave a wave's loads one after the other.  us, one wave a row and
// four, 2880 bf16 and 4436 float32 columns: 40 rows 6.1 / 5.0 and 16.8 / 7.0, 1200
// 10.6 / 7.0 and 26.8 / 14.5, 4000 14.4 / 15.0 and 37.5 / 36.1, 8000 21.7 / 25.9 and
// 61.2 / 65.8.
constexpr int kSplitRows = 2048;

// W waves per routed row: dys[pos] = w dout[t], dw = <dout[t], ys[pos]>.
template <typename DT, int N, int W>
__global__ __launch_bounds__(kThreads) void k_combine_backward(
    OrderShape s, const DT *__restrict__ dout, const DT *__restrict__ ys,
    const int *__restrict__ row_pos, const float *__restrict__ w, DT *__restrict__ dys,
    float *__restrict__ dw) {
  constexpr int BYTES = sizeof(DT) * N;
  __shared__ float part[kWaves];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int p = __builtin_amdgcn_readfirstlane((blockIdx.x * kWaves + wave) / W);
  if (p >= s.R) return;
  const int pos = row_pos[p], H = s.H, share = wave % W;
  if ((unsigned)pos >= (unsigned)s.R) {
    if (dw && lane == 0 && share == 0) dw[p] = 0.f;
    return;
  }
  const float g = w ? w[p] : 1.f;
  const DT *d = dout + (size_t)(p / s.k) * H;
  const size_t row = (size_t)pos * H;
  float sum = 0.f;
  for (int c = (share * kWave + lane) * N; c < H; c += W * kWave * N) {
    const int at = min(c, H - N);
    float a[N], o[N];
    unpack<DT, N>(*raw<BYTES>(d + at), a);
    if (dw) {
      float y[N];
      unpack<DT, N>(__builtin_nontemporal_load(raw<BYTES>(ys + row + at)), y);
      // (the last chunk's elements that the one before it has counted stay out)
#pragma unroll
      for (int i = 0; i < N; ++i) sum = at + i >= c ? fmaf(a[i], y[i], sum) : sum;
    }
    if (dys) {
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = g * a[i];
      // (the wave's lanes share c - lane N)
      store_past<BYTES>(pack<DT, N>(o), reinterpret_cast<char *>(dys + row), at * sizeof(DT),
                        (c - lane * N) * sizeof(DT), min(c - lane * N + kWave * N, H) * sizeof(DT));
    }
  }
  if (dw) {
#pragma unroll
    for (int m = kWave / 2; m > 0; m >>= 1) sum += __shfl_xor(sum, m);
    if constexpr (W > 1) {  // (W = kWaves: the row is the workgroup's)
      if (lane == 0) part[wave] = sum;
      __syncthreads();
      sum = part[0];
#pragma unroll
      for (int q = 1; q < W; ++q) sum += part[q];
    }
    if (lane == 0 && share == 0) dw[p] = sum;
  }
}

template <int BYTES>
hipError_t dispatch_t(const OrderShape &s, int row_bytes, const void *x, const int *ids,
                      int *expert_start, int *sorted_rows, int *row_pos, void *xs, int *counts,
                      hipStream_t st) {
  const char *cx = static_cast<const char *>(x);
  char *cxs = static_cast<char *>(xs);
  if (s.R <= kFusedRows)
    return launch_kernel(k_dispatch_fused<BYTES>, dim3(s.R + 1), dim3(kThreads), 0, st, s, row_bytes,
                         cx, ids, expert_start, sorted_rows, row_pos, cxs);
  const int C = order_chunk_rows(s.R), nch = order_chunks(s.R);
  int bits = 0;
  while ((1 << bits) < s.E) ++bits;
  hipError_t e;
  if (counts_itself(s.R, s.E)) {
    e = launch_kernel(k_order_place<true>, dim3(nch), dim3(kThreads), 0, st, s.R, s.E, C, nch, bits, 8, ids,
                      static_cast<const int *>(nullptr), expert_start, sorted_rows, row_pos);
  } else {
    e = launch_kernel(k_order_count, dim3(nch), dim3(kThreads), 0, st, s.R, s.E, C, ids, counts);
    if (e != hipSuccess) return e;
    e = launch_kernel(k_order_place<false>, dim3(nch), dim3(kThreads), 0, st, s.R, s.E, C, nch, bits,
                      bits < 8 ? bits : 8, ids, static_cast<const int *>(counts), expert_start, sorted_rows,
                      row_pos);
  }
  if (e != hipSuccess || !xs) return e;
  const RowGrid g = row_grid(s.T, (row_bytes + BYTES - 1) / BYTES);
  return launch_kernel(k_scatter<BYTES>, g.grid, dim3(kThreads), 0, st, s, row_bytes, g.tpt_shift, cx,
                       static_cast<const int *>(row_pos), cxs);
}

template <typename DT, int N>
hipError_t combine_t(const OrderShape &s, const void *ys, const int *row_pos, const float *w, void *out,
                     hipStream_t st) {
  const RowGrid g = row_grid(s.T, (s.H + N - 1) / N);
  if (w)
    return launch_kernel(k_combine_order<DT, N, true>, g.grid, dim3(kThreads), 0, st, s, g.tpt_shift,
                         static_cast<const DT *>(ys), row_pos, w, static_cast<DT *>(out));
  return launch_kernel(k_combine_order<DT, N, false>, g.grid, dim3(kThreads), 0, st, s, g.tpt_shift,
                       static_cast<const DT *>(ys), row_pos, w, static_cast<DT *>(out));
}

template <typename DT, int N>
hipError_t combine_backward_t(const OrderShape &s, const void *dout, const void *ys, const int *row_pos,
                              const float *w, void *dys, float *dw, hipStream_t st) {
  auto run = [&](auto kern, int W) {
    return launch_kernel(kern, dim3(((long long)s.R * W + kWaves - 1) / kWaves), dim3(kThreads), 0, st, s,
                         static_cast<const DT *>(dout), static_cast<const DT *>(ys), row_pos, w,
                         static_cast<DT *>(dys), dw);
  };
  if (s.R <= kSplitRows) return run(k_combine_backward<DT, N, kWaves>, kWaves);
  return run(k_combine_backward<DT, N, 1>, 1);
}

}  // namespace

int dispatch_counts(int R, int E) { return R <= kFusedRows || counts_itself(R, E) ? 0 : order_chunks(R); }

// 16 bytes a lane, or an element where a row is shorter than that.
hipError_t launch_dispatch(const OrderShape &s, const void *x, const int *ids, int *expert_start,
                           int *sorted_rows, int *row_pos, void *xs, int *counts, hipStream_t st) {
  const int b = s.H * (s.bf16 ? 2 : 4);
  if (b >= 16) return dispatch_t<16>(s, b, x, ids, expert_start, sorted_rows, row_pos, xs, counts, st);
  return dispatch_t<2>(s, b, x, ids, expert_start, sorted_rows, row_pos, xs, counts, st);
}

hipError_t launch_combine_rows(const OrderShape &s, const void *ys, const int *row_pos, const float *w,
                               void *out, hipStream_t st) {
  if (s.bf16)
    return s.H >= 8 ? combine_t<uint16_t, 8>(s, ys, row_pos, w, out, st)
                    : combine_t<uint16_t, 1>(s, ys, row_pos, w, out, st);
  return s.H >= 4 ? combine_t<float, 4>(s, ys, row_pos, w, out, st)
                  : combine_t<float, 1>(s, ys, row_pos, w, out, st);
}

hipError_t launch_combine_backward(const OrderShape &s, const void *dout, const void *ys,
                                   const int *row_pos, const float *w, void *dys, float *dw,
                                   hipStream_t st) {
  if (s.bf16)
    return s.H >= 8 ? combine_backward_t<uint16_t, 8>(s, dout, ys, row_pos, w, dys, dw, st)
                    : combine_backward_t<uint16_t, 1>(s, dout, ys, row_pos, w, dys, dw, st);
  return s.H >= 4 ? combine_backward_t<float, 4>(s, dout, ys, row_pos, w, dys, dw, st)
                  : combine_backward_t<float, 1>(s, dout, ys, row_pos, w, dys, dw, st);
}

}  // namespace moelora
