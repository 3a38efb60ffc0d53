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

}  // extern "C"
