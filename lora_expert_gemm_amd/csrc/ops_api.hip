// C entry points of the stand-alone operators: argument checks, then one to
// three launches on the caller's stream.  No entry point allocates,
// synchronises or keeps anything between calls.
#include <algorithm>
#include <atomic>
#include <cstdio>
#include <mutex>

#include "../../include/moelora.h"
#include "kernels.h"
#include "ops.h"

using namespace moelora;

namespace {

constexpr int kMaxE = 1024, kMaxK = 32, kMaxWidth = 65536, kMaxOut = 131072, kMaxMats = 65535;
constexpr long long kMaxRows = 1ll << 24;

bool ok16(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool opt16(const void *p) { return !p || ok16(p); }

moelora_status from_hip(hipError_t e) { return e == hipSuccess ? MOELORA_OK : MOELORA_ERR_HIP; }

// Load, on the current device, every kernel these operators can launch, on
// the first call there: the launchers run once per variant with
// tl_resolve_only set, so that no later call loads code.  No pointer is read.
hipError_t resolve_all() {
  void *const f = reinterpret_cast<void *>(uintptr_t{1} << 12);
  int *const fi = static_cast<int *>(f);
  float *const ff = static_cast<float *>(f);
  uint8_t *const fb = static_cast<uint8_t *>(f);
  hipError_t e = hipSuccess;
  auto need = [&](hipError_t r) {
    if (e == hipSuccess) e = r;
  };
  for (int bf16 = 0; bf16 < 2; ++bf16) {
    for (int H : {8, 1}) {  // rows of 16 bytes and more, and shorter ones
      for (int R : {1, 4096, 1 << 20}) {
        const OrderShape s{R, H, 1, 1, R, bf16 != 0};
        need(launch_dispatch(s, f, fi, fi, fi, fi, f, fi, nullptr));
        need(launch_combine_rows(s, f, fi, ff, f, nullptr));
        need(launch_combine_rows(s, f, fi, nullptr, f, nullptr));
        need(launch_combine_backward(s, f, f, fi, ff, f, ff, nullptr));
      }
    }
    need(launch_quantize_rows(QuantRowsArgs{f, nullptr, fb, ff, 1, 1, 1, 1}, bf16, nullptr));
    need(launch_quantize_weights(QuantWeightsArgs{f, fb, nullptr, ff, nullptr, 1, 1, 1}, bf16, nullptr));
    for (int silu = 0; silu < 2; ++silu) need(resolve_fp8_gemm(silu, bf16));
    for (int E : {16, 32, 64, 128, 256, 512, 1024}) {  // one of each of the router's forms
      const RouterArgs r{f, nullptr, 1, E, 1};
      for (int all = 0; all < 2; ++all) {
        need(launch_route(r, all, bf16, fi, ff, nullptr));
        need(launch_route_backward(r, RouteGradArgs{fi, ff, ff, fi, ff, f}, all, bf16, nullptr));
      }
      need(launch_balance(r, bf16, fi, BalanceOut{fi, ff, ff}, f, nullptr));
    }
    const Fp4WeightsArgs w{f, fb, f, fb, fb, 1, 1, 1, 1, 1, 1};
    need(launch_quantize_fp4(w, bf16, nullptr));
    need(launch_pack_fp4(w, nullptr));
    need(launch_dequantize_fp4(w, bf16, nullptr));
    for (int silu = 0; silu < 2; ++silu) need(resolve_fp4_gemm(silu, bf16));
  }
  return e;
}

moelora_status resolve_once() {
  static std::atomic<uint64_t> done{0};
  static std::mutex mu;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return MOELORA_ERR_HIP;
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return MOELORA_OK;
  std::lock_guard<std::mutex> lock(mu);
  if (bit && (done.load(std::memory_order_acquire) & bit)) return MOELORA_OK;
  tl_resolve_only = true;
  const hipError_t e = resolve_all();
  tl_resolve_only = false;
  if (e != hipSuccess) return MOELORA_ERR_HIP;
  if (bit) done.fetch_or(bit, std::memory_order_acq_rel);
  return MOELORA_OK;
}

// After every host-side check: kernels resolved, and no error pending from
// an earlier call.
moelora_status ready() {
  const moelora_status st = resolve_once();
  if (st == MOELORA_OK) (void)hipGetLastError();
  return st;
}

// Shape checks shared by the token-order operators.
moelora_status order_shape(int32_t T, int32_t H, int32_t E, int32_t k, int32_t dtype, OrderShape *s) {
  if (T < 0) return MOELORA_ERR_INVALID_ARG;
  if (H < 1 || H > kMaxWidth || E < 1 || E > kMaxE || k < 1 || k > kMaxK || (long long)T * k > kMaxRows ||
      (dtype != MOELORA_F32 && dtype != MOELORA_BF16))
    return MOELORA_ERR_UNSUPPORTED;
  *s = OrderShape{T, H, E, k, T * k, dtype == MOELORA_BF16};
  return MOELORA_OK;
}

// Sizes of the product; the pointers are left null.
moelora_status gemm_shape(int32_t n_rows, int32_t n_out, int32_t width, int32_t n_experts, int32_t out_dtype,
                          uint32_t flags, Fp8GemmArgs *a) {
  if (n_rows < 0) return MOELORA_ERR_INVALID_ARG;
  if (n_rows > kMaxRows || n_out < 1 || n_out > kMaxOut || width < 1 || width > kMaxWidth ||
      n_experts < 1 || n_experts > kMaxE || (flags & ~MOELORA_FP8_SILU_MUL) ||
      (out_dtype != MOELORA_F32 && out_dtype != MOELORA_BF16))
    return MOELORA_ERR_UNSUPPORTED;
  a->R = n_rows;
  a->N = n_out;
  a->K = width;
  a->E = n_experts;
  a->KB = (width + 127) / 128;
  a->NB = (n_out + 127) / 128;
  a->P = row_pitch8(width);
  return MOELORA_OK;
}

// Sizes of the router's operators; the pointers are left null.
moelora_status router_shape(int32_t T, int32_t E, int32_t k, int32_t dtype, RouterArgs *a) {
  if (T < 0) return MOELORA_ERR_INVALID_ARG;
  if (E < 1 || E > kMaxE || k < 1 || k > kMaxK || k > E || (long long)T * k > kMaxRows ||
      (dtype != MOELORA_F32 && dtype != MOELORA_BF16))
    return MOELORA_ERR_UNSUPPORTED;
  *a = RouterArgs{nullptr, nullptr, T, E, k};
  return MOELORA_OK;
}

// A launch holds fewer than 2^32 threads; a workgroup of 256 makes four fours of tiles.
constexpr long long kMaxTileFours = (1ll << 26) - 4;
// Sizes of 4-bit weights; the pointers are left null.
moelora_status fp4_shape(int32_t mats, int32_t N, int32_t K, Fp4WeightsArgs *a) {
  if (mats < 0) return MOELORA_ERR_INVALID_ARG;
  if (mats > kMaxMats || N < 1 || N > kMaxOut || K < 1 || K > kMaxWidth) return MOELORA_ERR_UNSUPPORTED;
  a->mats = mats;
  a->N = N;
  a->K = K;
  a->NT = (N + 15) / 16;
  a->KB = (K + 127) / 128;
  a->KQ = (a->KB + 3) / 4;
  return (long long)mats * a->NT * a->KQ <= kMaxTileFours ? MOELORA_OK : MOELORA_ERR_UNSUPPORTED;
}

constexpr long long kMaxResults = 1ll << 34;  // (a thread of a tile makes eight and more)
// Sizes of the product on 4-bit weights; the pointers are left null.
moelora_status fp4_gemm_shape(int32_t n_rows, int32_t n_out, int32_t width, int32_t n_experts, int32_t dtype,
                              uint32_t flags, Fp4GemmArgs *a) {
  if (n_rows < 0) return MOELORA_ERR_INVALID_ARG;
  if (n_rows > kMaxRows || n_experts < 1 || n_experts > kMaxE || (flags & ~MOELORA_FP4_SILU_MUL) ||
      (dtype != MOELORA_F32 && dtype != MOELORA_BF16))
    return MOELORA_ERR_UNSUPPORTED;
  Fp4WeightsArgs w{};
  if ((long long)n_rows * n_out > kMaxResults) return MOELORA_ERR_UNSUPPORTED;
  const moelora_status st = fp4_shape(n_experts * (flags & MOELORA_FP4_SILU_MUL ? 2 : 1), n_out, width, &w);
  *a = Fp4GemmArgs{};
  a->R = n_rows;
  a->N = n_out;
  a->K = width;
  a->E = n_experts;
  a->NT = w.NT;
  a->KB = w.KB;
  a->KQ = w.KQ;
  return st;
}

size_t dispatch_ws(const OrderShape &s) { return dispatch_counts(s.R, s.E) * (size_t)s.E * 4; }
// What a caller is told to keep: enough for every smaller batch as well (past
// kOrderChunks full chunks the chunks grow and their number falls back).
size_t dispatch_ws_upto(const OrderShape &s) {
  const int full = std::min((s.R + kOrderMinRows - 1) / kOrderMinRows, kOrderChunks);
  return dispatch_counts(s.R, s.E) ? full * (size_t)s.E * 4 : 0;
}

}  // namespace

extern "C" {

moelora_status moelora_dispatch_workspace(int32_t n_tokens, int32_t n_experts, int32_t top_k,
                                          size_t *workspace_bytes) {
  if (!workspace_bytes) return MOELORA_ERR_INVALID_ARG;
  OrderShape s;
  const moelora_status st = order_shape(n_tokens, 1, n_experts, top_k, MOELORA_F32, &s);
  if (st == MOELORA_OK) *workspace_bytes = dispatch_ws_upto(s);
  return st;
}

moelora_status moelora_dispatch(int32_t n_tokens, int32_t hidden, int32_t n_experts, int32_t top_k,
                                int32_t dtype, const void *x, const int32_t *topk_ids,
                                int32_t *expert_start, int32_t *sorted_rows, int32_t *row_pos, void *xs,
                                void *workspace, size_t workspace_bytes, moelora_stream_t stream) {
  OrderShape s;
  moelora_status st = order_shape(n_tokens, hidden, n_experts, top_k, dtype, &s);
  if (st != MOELORA_OK) return st;
  if (!ok16(expert_start)) return MOELORA_ERR_INVALID_ARG;
  if (s.R > 0 && (!ok16(topk_ids) || !ok16(sorted_rows) || !ok16(row_pos) || !opt16(xs) || !opt16(x) ||
                  (xs && !x)))
    return MOELORA_ERR_INVALID_ARG;
  const size_t need = dispatch_ws(s);
  if (need > 0 && !ok16(workspace)) return MOELORA_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MOELORA_ERR_WORKSPACE;
  if ((st = ready()) != MOELORA_OK) return st;
  return from_hip(launch_dispatch(s, x, topk_ids, expert_start, sorted_rows, row_pos, xs,
                                  static_cast<int *>(workspace), reinterpret_cast<hipStream_t>(stream)));
}

moelora_status moelora_dispatch_backward(int32_t n_tokens, int32_t hidden, int32_t top_k, int32_t dtype,
                                         const void *dxs, const int32_t *row_pos, void *dx,
                                         moelora_stream_t stream) {
  OrderShape s;
  moelora_status st = order_shape(n_tokens, hidden, 1, top_k, dtype, &s);
  if (st != MOELORA_OK || s.R == 0) return st;
  if (!ok16(dxs) || !ok16(row_pos) || !ok16(dx)) return MOELORA_ERR_INVALID_ARG;
  if ((st = ready()) != MOELORA_OK) return st;
  return from_hip(launch_combine_rows(s, dxs, row_pos, nullptr, dx, reinterpret_cast<hipStream_t>(stream)));
}

moelora_status moelora_combine(int32_t n_tokens, int32_t hidden, int32_t top_k, int32_t dtype,
                               const void *ys, const int32_t *row_pos, const float *topk_w, void *out,
                               moelora_stream_t stream) {
  OrderShape s;
  moelora_status st = order_shape(n_tokens, hidden, 1, top_k, dtype, &s);
  if (st != MOELORA_OK || s.R == 0) return st;
  if (!ok16(ys) || !ok16(row_pos) || !ok16(topk_w) || !ok16(out)) return MOELORA_ERR_INVALID_ARG;
  if ((st = ready()) != MOELORA_OK) return st;
  return from_hip(launch_combine_rows(s, ys, row_pos, topk_w, out, reinterpret_cast<hipStream_t>(stream)));
}

moelora_status moelora_combine_backward(int32_t n_tokens, int32_t hidden, int32_t top_k, int32_t dtype,
                                        const void *dout, const void *ys, const int32_t *row_pos,
                                        const float *topk_w, void *dys, float *dw,
                                        moelora_stream_t stream) {
  OrderShape s;
  moelora_status st = order_shape(n_tokens, hidden, 1, top_k, dtype, &s);
  if (st != MOELORA_OK || s.R == 0) return st;
  if (!ok16(dout) || !ok16(row_pos) || (!dys && !dw) || !opt16(ys) || !opt16(topk_w) || !opt16(dys) ||
      !opt16(dw) || (dys && !topk_w) || (dw && !ys))
    return MOELORA_ERR_INVALID_ARG;
  if ((st = ready()) != MOELORA_OK) return st;
  return from_hip(launch_combine_backward(s, dout, ys, row_pos, topk_w, dys, dw,
                                          reinterpret_cast<hipStream_t>(stream)));
}

moelora_status moelora_quantize_rows(int32_t n_rows, int32_t width, int32_t dtype, const void *x,
                                     int32_t n_src, const int32_t *rows, int32_t row_div, void *codes,
                                     float *scales, moelora_stream_t stream) {
  if (n_rows < 0 || n_src < 0 || row_div < 1 || (!rows && (n_src < n_rows || row_div != 1)))
    return MOELORA_ERR_INVALID_ARG;
  if (width < 1 || width > kMaxWidth || n_rows > kMaxRows || n_src > kMaxRows ||
      (dtype != MOELORA_F32 && dtype != MOELORA_BF16))
    return MOELORA_ERR_UNSUPPORTED;
  if (n_rows == 0) return MOELORA_OK;
  if ((n_src > 0 && !ok16(x)) || !opt16(rows) || !ok16(codes) || !ok16(scales))
    return MOELORA_ERR_INVALID_ARG;
  const moelora_status st = ready();
  if (st != MOELORA_OK) return st;
  return from_hip(launch_quantize_rows(
      QuantRowsArgs{x, rows, static_cast<uint8_t *>(codes), scales, n_rows, width, n_src, row_div},
      dtype == MOELORA_BF16, reinterpret_cast<hipStream_t>(stream)));
}

moelora_status moelora_quantize_weights(int32_t n_mats, int32_t rows, int32_t width, int32_t dtype,
                                        const void *w, void *codes, float *scales, void *codes_t,
                                        float *scales_t, moelora_stream_t stream) {
  if (n_mats < 0) return MOELORA_ERR_INVALID_ARG;
  if (n_mats > kMaxMats || rows < 1 || rows > kMaxOut || width < 1 || width > kMaxWidth ||
      (dtype != MOELORA_F32 && dtype != MOELORA_BF16))
    return MOELORA_ERR_UNSUPPORTED;
  if (n_mats == 0) return MOELORA_OK;
  if (!ok16(w) || !ok16(codes) || !ok16(scales) || !opt16(codes_t) || !opt16(scales_t) ||
      !codes_t != !scales_t)
    return MOELORA_ERR_INVALID_ARG;
  const moelora_status st = ready();
  if (st != MOELORA_OK) return st;
  return from_hip(launch_quantize_weights(
      QuantWeightsArgs{w, static_cast<uint8_t *>(codes), static_cast<uint8_t *>(codes_t), scales, scales_t,
                       n_mats, rows, width},
      dtype == MOELORA_BF16, reinterpret_cast<hipStream_t>(stream)));
}

moelora_status moelora_fp8_gemm(int32_t n_rows, int32_t n_out, int32_t width, int32_t n_experts,
                                int32_t out_dtype, uint32_t flags, const void *codes, const float *scales,
                                const int32_t *expert_start, const void *w_codes, const float *w_scales,
                                void *out, moelora_stream_t stream) {
  Fp8GemmArgs a{};
  moelora_status st = gemm_shape(n_rows, n_out, width, n_experts, out_dtype, flags, &a);
  if (st != MOELORA_OK || n_rows == 0) return st;
  if (!ok16(codes) || !ok16(scales) || !opt16(expert_start) || !ok16(w_codes) || !ok16(w_scales) ||
      !ok16(out) || (!expert_start && n_experts != 1))
    return MOELORA_ERR_INVALID_ARG;
  if ((st = ready()) != MOELORA_OK) return st;
  a.x = static_cast<const uint8_t *>(codes);
  a.xs = scales;
  a.start = expert_start;
  a.w = static_cast<const uint8_t *>(w_codes);
  a.ws = w_scales;
  a.out = out;
  return from_hip(launch_fp8_gemm(a, flags & MOELORA_FP8_SILU_MUL, out_dtype == MOELORA_BF16,
                                  reinterpret_cast<hipStream_t>(stream)));
}

moelora_status moelora_fp8_gemm_info(int32_t n_rows, int32_t n_out, int32_t width, int32_t n_experts,
                                     int32_t out_dtype, uint32_t flags, char *buf, size_t buf_len) {
  Fp8GemmArgs a{};
  const moelora_status st = gemm_shape(n_rows, n_out, width, n_experts, out_dtype, flags, &a);
  if (st != MOELORA_OK) return st;
  if (!buf || buf_len == 0) return MOELORA_ERR_INVALID_ARG;
  if (n_rows == 0) {
    snprintf(buf, buf_len, "kernel=none");
    return MOELORA_OK;
  }
  const Fp8Choice c = choose_fp8_gemm(a, flags & MOELORA_FP8_SILU_MUL, out_dtype == MOELORA_BF16);
  const char *name = "";
  switch (c.kernel) {
    case Fp8Kernel::kStream1Once: name = "stream1_once"; break;
    case Fp8Kernel::kStream1: name = "stream1"; break;
    case Fp8Kernel::kStream2: name = "stream2"; break;
    case Fp8Kernel::kTile2x2Once: name = "tile2x2_once"; break;
    case Fp8Kernel::kTile2x2: name = "tile2x2"; break;
    case Fp8Kernel::kTile2x4Once: name = "tile2x4_once"; break;
    case Fp8Kernel::kTile2x4: name = "tile2x4"; break;
    case Fp8Kernel::kTile2x8: name = "tile2x8"; break;
    case Fp8Kernel::kTile4x8: name = "tile4x8"; break;
    case Fp8Kernel::kTile4x4: name = "tile4x4"; break;
  }
  snprintf(buf, buf_len, "kernel=%s groups=%d", name, c.groups);
  return MOELORA_OK;
}

moelora_status moelora_route(int32_t n_tokens, int32_t n_experts, int32_t top_k, int32_t dtype, uint32_t flags,
                             const void *logits, const uint8_t *token_mask, int32_t *topk_ids, float *topk_w,
                             moelora_stream_t stream) {
  RouterArgs a;
  moelora_status st = router_shape(n_tokens, n_experts, top_k, dtype, &a);
  if (st != MOELORA_OK) return st;
  if (flags & ~MOELORA_ROUTE_SOFTMAX_ALL) return MOELORA_ERR_UNSUPPORTED;
  if (n_tokens == 0) return MOELORA_OK;
  if (!ok16(logits) || !opt16(token_mask) || !ok16(topk_ids) || !ok16(topk_w)) return MOELORA_ERR_INVALID_ARG;
  if ((st = ready()) != MOELORA_OK) return st;
  a.logits = logits;
  a.mask = token_mask;
  return from_hip(launch_route(a, flags & MOELORA_ROUTE_SOFTMAX_ALL, dtype == MOELORA_BF16, topk_ids, topk_w,
                               reinterpret_cast<hipStream_t>(stream)));
}

moelora_status moelora_balance_loss_workspace(int32_t n_tokens, int32_t n_experts, int32_t top_k,
                                              size_t *workspace_bytes) {
  if (!workspace_bytes) return MOELORA_ERR_INVALID_ARG;
  RouterArgs a;
  const moelora_status st = router_shape(n_tokens, n_experts, top_k, MOELORA_F32, &a);
  if (st == MOELORA_OK) *workspace_bytes = balance_workspace(a.T, a.E);
  return st;
}

moelora_status moelora_balance_loss(int32_t n_tokens, int32_t n_experts, int32_t top_k, int32_t dtype,
                                    const void *logits, const uint8_t *token_mask, const int32_t *topk_ids,
                                    int32_t *counts, float *prob_sum, float *loss, void *workspace,
                                    size_t workspace_bytes, moelora_stream_t stream) {
  RouterArgs a;
  moelora_status st = router_shape(n_tokens, n_experts, top_k, dtype, &a);
  if (st != MOELORA_OK) return st;
  if (!ok16(counts) || !ok16(prob_sum) || !ok16(loss)) return MOELORA_ERR_INVALID_ARG;
  if (n_tokens > 0 && (!ok16(logits) || !opt16(token_mask) || !ok16(topk_ids))) return MOELORA_ERR_INVALID_ARG;
  const size_t need = balance_workspace(a.T, a.E);
  if (need > 0 && !ok16(workspace)) return MOELORA_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MOELORA_ERR_WORKSPACE;
  if ((st = ready()) != MOELORA_OK) return st;
  a.logits = logits;
  a.mask = token_mask;
  return from_hip(launch_balance(a, dtype == MOELORA_BF16, topk_ids, BalanceOut{counts, prob_sum, loss}, workspace,
                                 reinterpret_cast<hipStream_t>(stream)));
}

moelora_status moelora_route_backward(int32_t n_tokens, int32_t n_experts, int32_t top_k, int32_t dtype,
                                      uint32_t flags, const void *logits, const uint8_t *token_mask,
                                      const int32_t *topk_ids, const float *topk_w, const float *dtopk_w,
                                      const int32_t *counts, const float *dloss, void *dlogits,
                                      moelora_stream_t stream) {
  RouterArgs a;
  moelora_status st = router_shape(n_tokens, n_experts, top_k, dtype, &a);
  if (st != MOELORA_OK) return st;
  if (flags & ~MOELORA_ROUTE_SOFTMAX_ALL) return MOELORA_ERR_UNSUPPORTED;
  if (n_tokens == 0) return MOELORA_OK;
  if (!ok16(logits) || !opt16(token_mask) || !opt16(topk_ids) || !opt16(topk_w) || !opt16(dtopk_w) ||
      !opt16(counts) || !opt16(dloss) || !ok16(dlogits) || (!dtopk_w && !counts) || !counts != !dloss ||
      (dtopk_w && (!topk_ids || !topk_w)))
    return MOELORA_ERR_INVALID_ARG;
  if ((st = ready()) != MOELORA_OK) return st;
  a.logits = logits;
  a.mask = token_mask;
  return from_hip(launch_route_backward(a, RouteGradArgs{topk_ids, topk_w, dtopk_w, counts, dloss, dlogits},
                                        flags & MOELORA_ROUTE_SOFTMAX_ALL, dtype == MOELORA_BF16,
                                        reinterpret_cast<hipStream_t>(stream)));
}

moelora_status moelora_quantize_weights_fp4(int32_t n_mats, int32_t rows, int32_t width, int32_t dtype,
                                            const void *w, void *codes, void *scales, moelora_stream_t stream) {
  Fp4WeightsArgs a{};
  moelora_status st = fp4_shape(n_mats, rows, width, &a);
  if (st != MOELORA_OK) return st;
  if (dtype != MOELORA_F32 && dtype != MOELORA_BF16) return MOELORA_ERR_UNSUPPORTED;
  if (n_mats == 0) return MOELORA_OK;
  if (!ok16(w) || !ok16(codes) || !ok16(scales)) return MOELORA_ERR_INVALID_ARG;
  if ((st = ready()) != MOELORA_OK) return st;
  a.src = w;
  a.codes = static_cast<uint8_t *>(codes);
  a.scales = static_cast<uint8_t *>(scales);
  return from_hip(launch_quantize_fp4(a, dtype == MOELORA_BF16, reinterpret_cast<hipStream_t>(stream)));
}

moelora_status moelora_pack_weights_fp4(int32_t n_mats, int32_t rows, int32_t width, const void *row_codes,
                                        const void *row_scales, void *codes, void *scales,
                                        moelora_stream_t stream) {
  Fp4WeightsArgs a{};
  moelora_status st = fp4_shape(n_mats, rows, width, &a);
  if (st != MOELORA_OK || n_mats == 0) return st;
  if (!ok16(row_codes) || !ok16(row_scales) || !ok16(codes) || !ok16(scales)) return MOELORA_ERR_INVALID_ARG;
  if ((st = ready()) != MOELORA_OK) return st;
  a.src = row_codes;
  a.src_scales = static_cast<const uint8_t *>(row_scales);
  a.codes = static_cast<uint8_t *>(codes);
  a.scales = static_cast<uint8_t *>(scales);
  return from_hip(launch_pack_fp4(a, reinterpret_cast<hipStream_t>(stream)));
}

moelora_status moelora_dequantize_weights_fp4(int32_t n_mats, int32_t rows, int32_t width, int32_t dtype,
                                              const void *codes, const void *scales, void *w,
                                              moelora_stream_t stream) {
  Fp4WeightsArgs a{};
  moelora_status st = fp4_shape(n_mats, rows, width, &a);
  if (st != MOELORA_OK) return st;
  if (dtype != MOELORA_F32 && dtype != MOELORA_BF16) return MOELORA_ERR_UNSUPPORTED;
  if (n_mats == 0) return MOELORA_OK;
  if (!ok16(w) || !ok16(codes) || !ok16(scales)) return MOELORA_ERR_INVALID_ARG;
  if ((st = ready()) != MOELORA_OK) return st;
  a.dst = w;
  a.codes = static_cast<uint8_t *>(const_cast<void *>(codes));  // (read only on this way)
  a.scales = static_cast<uint8_t *>(const_cast<void *>(scales));
  return from_hip(launch_dequantize_fp4(a, dtype == MOELORA_BF16, reinterpret_cast<hipStream_t>(stream)));
}

moelora_status moelora_fp4_gemm(int32_t n_rows, int32_t n_out, int32_t width, int32_t n_experts, int32_t dtype,
                                uint32_t flags, const void *x, const int32_t *expert_start, const void *w_codes,
                                const void *w_scales, void *out, moelora_stream_t stream) {
  Fp4GemmArgs a;
  moelora_status st = fp4_gemm_shape(n_rows, n_out, width, n_experts, dtype, flags, &a);
  if (st != MOELORA_OK || n_rows == 0) return st;
  if (!ok16(x) || !opt16(expert_start) || !ok16(w_codes) || !ok16(w_scales) || !ok16(out) ||
      (!expert_start && n_experts != 1))
    return MOELORA_ERR_INVALID_ARG;
  if ((st = ready()) != MOELORA_OK) return st;
  a.x = x;
  a.start = expert_start;
  a.w = static_cast<const uint8_t *>(w_codes);
  a.ws = static_cast<const uint8_t *>(w_scales);
  a.out = out;
  return from_hip(launch_fp4_gemm(a, flags & MOELORA_FP4_SILU_MUL, dtype == MOELORA_BF16,
                                  reinterpret_cast<hipStream_t>(stream)));
}

moelora_status moelora_fp4_gemm_info(int32_t n_rows, int32_t n_out, int32_t width, int32_t n_experts,
                                     int32_t dtype, uint32_t flags, char *buf, size_t buf_len) {
  Fp4GemmArgs a;
  const moelora_status st = fp4_gemm_shape(n_rows, n_out, width, n_experts, dtype, flags, &a);
  if (st != MOELORA_OK) return st;
  if (!buf || buf_len == 0) return MOELORA_ERR_INVALID_ARG;
  if (n_rows == 0) {
    snprintf(buf, buf_len, "kernel=none");
    return MOELORA_OK;
  }
  static const char *const names[kFp4Kernels] = {"short",   "stream2",      "split1x1", "split2x2",     "tile4x2",
                                                 "tile4x1", "stream4_once", "tile2x2",  "tile4x2_once", "tile4x4",
                                                 "tile4x4_regs"};
  const Fp4Choice c = choose_fp4_gemm(a, flags & MOELORA_FP4_SILU_MUL, dtype == MOELORA_BF16);
  snprintf(buf, buf_len, "kernel=%s groups=%d", names[(int)c.kernel], c.groups);
  return MOELORA_OK;
}

}  // extern "C"
