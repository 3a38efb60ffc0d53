// Arguments and host-side launchers of the stand-alone operators: token
// order (dispatch / combine and their gradients), block-of-128 E4M3
// quantisation and the block-scaled product, the router with its losses, 4-bit
// weights and their product.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moelora {

// Routed rows p = t * k + j, R = T * k of them; rows of H elements, bf16 or float32.
struct OrderShape {
  int T, H, E, k, R;
  bool bf16;
};

// Chunks of the order of larger batches: 256 rows (64 a wave, one round of ballots:
// 1024 rows a chunk took 12.5 instead of 5 us for 25600), but at most
// kOrderChunks, so that every placing workgroup can add up the counts of the
// chunks before its own.
constexpr int kOrderChunks = 256, kOrderMinRows = 256;
inline int order_chunk_rows(int R) {
  const int c = (R + kOrderChunks - 1) / kOrderChunks;
  return (c + kOrderMinRows - 1) / kOrderMinRows * kOrderMinRows;
}
inline int order_chunks(int R) {
  const int c = order_chunk_rows(R);
  return c ? (R + c - 1) / c : 0;
}
// Chunks whose counts launch_dispatch writes (none where the ids are few enough
// to be counted where they are needed).
int dispatch_counts(int R, int E);

hipError_t launch_dispatch(const OrderShape &s, const void *x, const int *ids, int *expert_start,
                           int *sorted_rows, int *row_pos, void *xs, int *counts, hipStream_t st);
// out[t] = sum_j w[t][j] ys[row_pos[t][j]] (w null: 1)
hipError_t launch_combine_rows(const OrderShape &s, const void *ys, const int *row_pos, const float *w,
                               void *out, hipStream_t st);
hipError_t launch_combine_backward(const OrderShape &s, const void *dout, const void *ys,
                                   const int *row_pos, const float *w, void *dys, float *dw,
                                   hipStream_t st);

struct QuantRowsArgs {
  const void *x;
  const int *rows;  // null: row r of x
  uint8_t *codes;
  float *scales;
  int M, K, n_src, div;
};
hipError_t launch_quantize_rows(const QuantRowsArgs &a, bool bf16, hipStream_t st);

struct QuantWeightsArgs {
  const void *w;
  uint8_t *codes, *codes_t;  // codes_t, scales_t null: no transposed copy
  float *scales, *scales_t;
  int mats, N, K;
};
hipError_t launch_quantize_weights(const QuantWeightsArgs &a, bool bf16, hipStream_t st);

struct Fp8GemmArgs {
  const uint8_t *x;        // [R][P]
  const float *xs;         // [KB][R]
  const int *start;        // [E + 1], null with E = 1: all rows
  const uint8_t *w;        // [E][halves][N][P]
  const float *ws;         // [E][halves][NB][KB]
  void *out;               // [R][N]
  int R, N, K, E;
  int KB, NB;              // blocks of 128 along K and N
  size_t P;                // row pitch in bytes, KB * 128
};
// Which kernel a product takes: streamed, with 1 or 2 groups of 16 rows at a
// time and `groups` workgroups to share an expert's groups, or tiled, with
// weight tiles x token tiles of 16 a wave; Once: the weights go past the caches.
enum class Fp8Kernel {
  kStream1Once, kStream1, kStream2,
  kTile2x2Once, kTile2x2, kTile2x4Once, kTile2x4, kTile2x8, kTile4x8,  // (x8: bf16 results)
  kTile4x4,                                                           // float32 results
};
struct Fp8Choice {
  Fp8Kernel kernel;
  int groups;
};
Fp8Choice choose_fp8_gemm(const Fp8GemmArgs &a, bool silu, bool bf16);
hipError_t launch_fp8_gemm(const Fp8GemmArgs &a, bool silu, bool bf16, hipStream_t st);
// With tl_resolve_only set: looks up every kernel launch_fp8_gemm can pick.
hipError_t resolve_fp8_gemm(bool silu, bool bf16);

// Router logits of T tokens over E experts, k picks each; mask null: every token.
struct RouterArgs {
  const void *logits;
  const uint8_t *mask;
  int T, E, k;
};
hipError_t launch_route(const RouterArgs &a, bool all, bool bf16, int *ids, float *w, hipStream_t st);

struct BalanceOut {
  int *counts;      // [E + 1]
  float *prob_sum;  // [E]
  float *loss;      // [2]
};
// Most workgroups whose sums launch_balance keeps in its workspace.
constexpr int kBalanceChunks = 256;
size_t balance_workspace(int T, int E);
hipError_t launch_balance(const RouterArgs &a, bool bf16, const int *ids, const BalanceOut &o, void *ws,
                          hipStream_t st);

struct RouteGradArgs {
  const int *ids;     // [T][k]
  const float *w;     // [T][k]
  const float *dw;    // [T][k], null: no gradient of the weights
  const int *counts;  // [E + 1], null: none of the losses
  const float *dloss; // [2]
  void *dlogits;
};
hipError_t launch_route_backward(const RouterArgs &a, const RouteGradArgs &q, bool all, bool bf16,
                                 hipStream_t st);

// 4-bit weights: mats matrices of N rows x K, in tiles of 16 x 128 (fp4.h).
struct Fp4WeightsArgs {
  const void *src;            // weights, or row-major codes
  const uint8_t *src_scales;  // row-major scales, with row-major codes
  void *dst;                  // values, for the way back
  uint8_t *codes, *scales;
  int mats, N, K;
  int NT, KB, KQ;  // tiles along N and K, fours of tiles along K
};
hipError_t launch_quantize_fp4(const Fp4WeightsArgs &a, bool bf16, hipStream_t st);
hipError_t launch_pack_fp4(const Fp4WeightsArgs &a, hipStream_t st);
hipError_t launch_dequantize_fp4(const Fp4WeightsArgs &a, bool bf16, hipStream_t st);

struct Fp4GemmArgs {
  const void *x;      // [R][K]
  const int *start;   // [E + 1], null with E = 1: all rows
  const uint8_t *w;   // [E][halves] matrices of codes
  const uint8_t *ws;  // ... and of scales
  void *out;          // [R][N]
  int R, N, K, E;
  int NT, KB, KQ;
};
// Which kernel a product takes.  Short: rows of less than 16 bytes.  Streamed:
// workgroups of 4 or 2 weight tiles (SILU: half of them gate), `groups` of them to
// share an expert's groups of 16 rows.  Split and tiled: weight tiles x token tiles of
// 16 a wave, split with the contraction over four groups of waves (Split2x2 of
// float32 rows: 4x1); Once: the weights go past the caches.
enum class Fp4Kernel {
  kShort, kStream2, kSplit1x1, kSplit2x2, kTile4x2,
  kTile4x1,                              // float32 rows
  kStream4Once, kTile2x2, kTile4x2Once, kTile4x4, kTile4x4Regs,  // bf16 rows (2x2, 4x4: whole 16 bytes, by DMA)
};
constexpr int kFp4Kernels = 11;
struct Fp4Choice {
  Fp4Kernel kernel;
  int groups;
};
Fp4Choice choose_fp4_gemm(const Fp4GemmArgs &a, bool silu, bool bf16);
hipError_t launch_fp4_gemm(const Fp4GemmArgs &a, bool silu, bool bf16, hipStream_t st);
// With tl_resolve_only set: looks up every kernel launch_fp4_gemm can pick.
hipError_t resolve_fp4_gemm(bool silu, bool bf16);

}  // namespace moelora
