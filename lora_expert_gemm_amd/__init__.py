"""Python binding of the MI355X (gfx950) fused MoE-LoRA layer library.

Thin ctypes marshalling over the C ABI of ``include/moelora.h``: every
function here has the name of the C entry point it calls and only converts
arguments (tensors to device pointers, status codes to exceptions).  All of
the layer's work runs in the library's HIP kernels; there is no fallback.
Importing this package fails loudly when ``_lib/libmoelora.so`` has not been
built (``python lora_expert_gemm_amd/build.py``).

Tensor arguments may be torch tensors (their ``data_ptr()`` is passed), raw
integer addresses, or None for a null pointer.
"""
import ctypes
import os
import re

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libmoelora.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "moelora.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the HIP library first "
        "(python lora_expert_gemm_amd/build.py)")

# One HIP runtime per process.  PyTorch for ROCm ships its own libamdhip64
# (requested by the unversioned name libamdhip64.so); this library requests
# libamdhip64.so.7.  Loaded after PyTorch, it binds to PyTorch's copy (same
# soname); loaded first, it would pull in ROCm's copy and PyTorch would then
# load a second runtime, and whichever initialises second finds no device.
# So PyTorch, when installed, is imported before the library is loaded.
try:
    import torch
except ImportError:
    torch = None

_lib = ctypes.CDLL(LIB_PATH)

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_HIP, ERR_DEVICE = 0, -1, -2, -3, -4, -5
ERR_TOO_LARGE = -6
STATIC_SCRATCH_BYTES = 64 << 20
F32, BF16, BF16_FP8W = 0, 1, 2
DEVERR_EXPERT_ID, DEVERR_ADAPTER_ID = 1, 2
FLAG_DETERMINISTIC, FLAG_DEBUG_CHECK_IDS = 1, 2
FP8_SILU_MUL = 1
N_STAGES = 6
STAGES = ("route_align", "shrink_gate_up", "gate_up", "shrink_down", "down", "combine")


class moelora_desc(ctypes.Structure):
    _fields_ = [("max_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("inter", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("n_adapters", ctypes.c_int32),
                ("rank", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class moelora_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("block_m", "cap", "nblk", "max_seg", "max_tiles", "reserved")] + \
               [(n, ctypes.c_size_t) for n in
                ("off_topk_ids", "off_topk_w", "off_sorted_rows", "off_block_expert",
                 "off_seg_start", "off_lora_seg", "off_tiles", "off_block_tile_start",
                 "off_counts", "off_error")]


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_lib.moelora_plan.argtypes = [ctypes.POINTER(moelora_desc), ctypes.POINTER(_P),
                              ctypes.POINTER(ctypes.c_size_t)]
_lib.moelora_plan.restype = ctypes.c_int
_lib.moelora_plan_destroy.argtypes = [_P]
_lib.moelora_plan_destroy.restype = None
_lib.moelora_forward.argtypes = [_P, _I32] + [_P] * 13 + [ctypes.c_size_t, _P]
_lib.moelora_forward.restype = ctypes.c_int
_lib.moelora_forward_noalloc.argtypes = [_P, _I32] + [_P] * 12 + [_P]
_lib.moelora_forward_noalloc.restype = ctypes.c_int
_lib.moelora_status_string.argtypes = [ctypes.c_int]
_lib.moelora_status_string.restype = ctypes.c_char_p
_lib.moelora_workspace_layout.argtypes = [_P, _I32, ctypes.POINTER(moelora_layout)]
_lib.moelora_workspace_layout.restype = ctypes.c_int
_lib.moelora_read_device_error.argtypes = [_P, _P, ctypes.POINTER(_I32), _P]
_lib.moelora_read_device_error.restype = ctypes.c_int
_lib.moelora_plan_info.argtypes = [_P, _I32, ctypes.c_char_p, ctypes.c_size_t]
_lib.moelora_plan_info.restype = ctypes.c_int
_lib.moelora_timing_begin.argtypes = [_P, _I32]
_lib.moelora_timing_begin.restype = ctypes.c_int
_lib.moelora_timing_end.argtypes = [_P, ctypes.POINTER(ctypes.c_double), _I32,
                                    ctypes.POINTER(_I32)]
_lib.moelora_timing_end.restype = ctypes.c_int
_U32 = ctypes.c_uint32
_lib.moelora_dispatch_workspace.argtypes = [_I32] * 3 + [ctypes.POINTER(ctypes.c_size_t)]
_lib.moelora_dispatch.argtypes = [_I32] * 5 + [_P] * 7 + [ctypes.c_size_t, _P]
_lib.moelora_dispatch_backward.argtypes = [_I32] * 4 + [_P] * 4
_lib.moelora_combine.argtypes = [_I32] * 4 + [_P] * 5
_lib.moelora_combine_backward.argtypes = [_I32] * 4 + [_P] * 7
_lib.moelora_quantize_rows.argtypes = [_I32] * 3 + [_P, _I32, _P, _I32] + [_P] * 3
_lib.moelora_quantize_weights.argtypes = [_I32] * 4 + [_P] * 6
_lib.moelora_fp8_gemm.argtypes = [_I32] * 5 + [_U32] + [_P] * 7
_lib.moelora_fp8_gemm_info.argtypes = [_I32] * 5 + [_U32, ctypes.c_char_p, ctypes.c_size_t]
for _n in ("dispatch_workspace", "dispatch", "dispatch_backward", "combine", "combine_backward",
           "quantize_rows", "quantize_weights", "fp8_gemm", "fp8_gemm_info"):
    getattr(_lib, "moelora_" + _n).restype = ctypes.c_int


def fp8_weight_buffer(codes, scales):
    """The weight-buffer layout of MOELORA_BF16_FP8W as a numpy uint8 array:
    the E4M3 codes ([E][rows][K] bytes), each row padded with zero bytes to a
    multiple of 128 bytes, zero bytes up to the next 256-byte boundary, then
    the float32 row scales ([E][rows])."""
    import numpy as np
    codes = np.asarray(codes, np.uint8)
    K = codes.shape[-1]
    pitch = (K + 127) // 128 * 128
    c = np.zeros(codes.shape[:-1] + (pitch,), np.uint8)
    c[..., :K] = codes
    c = c.reshape(-1)
    sc = np.ascontiguousarray(scales, np.float32).reshape(-1).view(np.uint8)
    off = (c.size + 255) // 256 * 256
    out = np.zeros(off + sc.size, np.uint8)
    out[:c.size] = c
    out[off:] = sc
    return out


class MoeLoraError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {moelora_status_string(status)} ({status})")


def _check(status, where):
    if status != OK:
        raise MoeLoraError(status, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def exported_symbols():
    """Names of the functions include/moelora.h declares."""
    with open(HEADER_PATH) as f:
        text = f.read()
    return sorted(set(re.findall(r"\b(moelora_[a-z0-9_]+)\s*\(", text)))


def moelora_status_string(status):
    return _lib.moelora_status_string(int(status)).decode()


def moelora_plan(max_tokens, hidden, inter, n_experts, top_k, n_adapters, rank,
                 dtype, flags=0):
    """-> (plan handle, workspace bytes)."""
    d = moelora_desc(max_tokens, hidden, inter, n_experts, top_k, n_adapters, rank,
                     dtype, flags)
    plan = _P()
    ws = ctypes.c_size_t()
    _check(_lib.moelora_plan(ctypes.byref(d), ctypes.byref(plan), ctypes.byref(ws)),
           "moelora_plan")
    return plan.value, ws.value


def moelora_plan_destroy(plan):
    _lib.moelora_plan_destroy(plan)


def moelora_forward(plan, n_tokens, x, router_logits, topk_ids, topk_w, adapter_ids,
                    w_gate_up, w_down, lora_a_gu, lora_b_gu, lora_a_d, lora_b_d,
                    out, workspace, workspace_bytes, stream=None):
    _check(_lib.moelora_forward(
        plan, n_tokens, _ptr(x), _ptr(router_logits), _ptr(topk_ids), _ptr(topk_w),
        _ptr(adapter_ids), _ptr(w_gate_up), _ptr(w_down), _ptr(lora_a_gu),
        _ptr(lora_b_gu), _ptr(lora_a_d), _ptr(lora_b_d), _ptr(out), _ptr(workspace),
        workspace_bytes, _stream(stream)), "moelora_forward")


def moelora_forward_noalloc(plan, n_tokens, x, router_logits, topk_ids, topk_w, adapter_ids,
                            w_gate_up, w_down, lora_a_gu, lora_b_gu, lora_a_d, lora_b_d,
                            out, stream=None):
    _check(_lib.moelora_forward_noalloc(
        plan, n_tokens, _ptr(x), _ptr(router_logits), _ptr(topk_ids), _ptr(topk_w),
        _ptr(adapter_ids), _ptr(w_gate_up), _ptr(w_down), _ptr(lora_a_gu),
        _ptr(lora_b_gu), _ptr(lora_a_d), _ptr(lora_b_d), _ptr(out), _stream(stream)),
        "moelora_forward_noalloc")


def moelora_workspace_layout(plan, n_tokens):
    lay = moelora_layout()
    _check(_lib.moelora_workspace_layout(plan, n_tokens, ctypes.byref(lay)),
           "moelora_workspace_layout")
    return {n: getattr(lay, n) for n, _ in moelora_layout._fields_}


def moelora_read_device_error(plan, workspace, stream=None):
    bits = _I32()
    _check(_lib.moelora_read_device_error(plan, _ptr(workspace), ctypes.byref(bits),
                                          _stream(stream)), "moelora_read_device_error")
    return bits.value


def moelora_plan_info(plan, n_tokens):
    buf = ctypes.create_string_buffer(512)
    _check(_lib.moelora_plan_info(plan, n_tokens, buf, len(buf)), "moelora_plan_info")
    return buf.value.decode()


def moelora_timing_begin(plan, max_calls):
    _check(_lib.moelora_timing_begin(plan, max_calls), "moelora_timing_begin")


def moelora_timing_end(plan):
    """-> (summed milliseconds per stage, number of timed forwards)."""
    ms = (ctypes.c_double * N_STAGES)()
    n = _I32()
    _check(_lib.moelora_timing_end(plan, ms, N_STAGES, ctypes.byref(n)), "moelora_timing_end")
    return list(ms), n.value


# ---- stand-alone operators.  A tensor argument is checked before its address
# is passed on: contiguous, on the current device, of the expected type (where
# bytes are expected, any type of one byte) and with at least as many elements
# as the call reads or writes.

_FLT, _BF, _INT = (torch.float32, torch.bfloat16, torch.int32) if torch else (None,) * 3
_BYTE = None


def _where(stream):
    """The stream to enqueue on (None: the current one) and the current device.
    (The stream's address by torch's raw getter where this torch has it: building
    a Stream object costs 2.7 us of host time, more than a small call's checks.)"""
    if torch is None:
        return _stream(stream), -1
    if stream is not None:
        dev = torch.cuda.current_device() if torch.cuda.is_available() else -1
        if isinstance(stream, torch.Stream) and stream.device_index != dev:
            raise ValueError(f"the stream is on device {stream.device_index}, not on the current device")
        return _stream(stream), dev
    dev = torch.cuda.current_device()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(dev) if raw else _stream(None), dev


def _buf(t, n, dtype, dev, name, optional=False):
    if t is None:
        if optional or n == 0:
            return None
        raise ValueError(f"{name} is required")
    if isinstance(t, int):
        return t
    if (t.numel() < n or not t.is_contiguous() or
            (t.itemsize != 1 if dtype is _BYTE else t.dtype is not dtype)):
        raise ValueError(f"{name}: expected a contiguous tensor of at least {n} elements of "
                         f"{dtype or 'one byte'}, got {tuple(t.shape)} {t.dtype} strides {t.stride()}")
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} is on {t.device}, not on the current device")
    return t.data_ptr()


def _dt(dtype):
    return _FLT if dtype == F32 else _BF


def moelora_dispatch_workspace(n_tokens, n_experts, top_k):
    """-> workspace bytes of moelora_dispatch."""
    n = ctypes.c_size_t()
    _check(_lib.moelora_dispatch_workspace(n_tokens, n_experts, top_k, ctypes.byref(n)),
           "moelora_dispatch_workspace")
    return n.value


def moelora_dispatch(n_tokens, hidden, n_experts, top_k, dtype, x, topk_ids, expert_start,
                     sorted_rows, row_pos, xs, workspace, workspace_bytes, stream=None):
    st, dev = _where(stream)
    R, dt = n_tokens * top_k, _dt(dtype)
    _check(_lib.moelora_dispatch(
        n_tokens, hidden, n_experts, top_k, dtype,
        _buf(x, n_tokens * hidden, dt, dev, "x", xs is None), _buf(topk_ids, R, _INT, dev, "topk_ids"),
        _buf(expert_start, n_experts + 1, _INT, dev, "expert_start"),
        _buf(sorted_rows, R, _INT, dev, "sorted_rows"), _buf(row_pos, R, _INT, dev, "row_pos"),
        _buf(xs, R * hidden, dt, dev, "xs", True),
        _buf(workspace, workspace_bytes, _BYTE, dev, "workspace", True), workspace_bytes,
        st), "moelora_dispatch")


def moelora_dispatch_backward(n_tokens, hidden, top_k, dtype, dxs, row_pos, dx, stream=None):
    st, dev = _where(stream)
    R, dt = n_tokens * top_k, _dt(dtype)
    _check(_lib.moelora_dispatch_backward(
        n_tokens, hidden, top_k, dtype, _buf(dxs, R * hidden, dt, dev, "dxs"),
        _buf(row_pos, R, _INT, dev, "row_pos"), _buf(dx, n_tokens * hidden, dt, dev, "dx"), st),
        "moelora_dispatch_backward")


def moelora_combine(n_tokens, hidden, top_k, dtype, ys, row_pos, topk_w, out, stream=None):
    st, dev = _where(stream)
    R, dt = n_tokens * top_k, _dt(dtype)
    _check(_lib.moelora_combine(
        n_tokens, hidden, top_k, dtype, _buf(ys, R * hidden, dt, dev, "ys"),
        _buf(row_pos, R, _INT, dev, "row_pos"), _buf(topk_w, R, _FLT, dev, "topk_w"),
        _buf(out, n_tokens * hidden, dt, dev, "out"), st), "moelora_combine")


def moelora_combine_backward(n_tokens, hidden, top_k, dtype, dout, ys, row_pos, topk_w, dys, dw,
                             stream=None):
    st, dev = _where(stream)
    R, dt = n_tokens * top_k, _dt(dtype)
    _check(_lib.moelora_combine_backward(
        n_tokens, hidden, top_k, dtype, _buf(dout, n_tokens * hidden, dt, dev, "dout"),
        _buf(ys, R * hidden, dt, dev, "ys", dw is None), _buf(row_pos, R, _INT, dev, "row_pos"),
        _buf(topk_w, R, _FLT, dev, "topk_w", dys is None), _buf(dys, R * hidden, dt, dev, "dys", True),
        _buf(dw, R, _FLT, dev, "dw", True), st), "moelora_combine_backward")


def moelora_quantize_rows(n_rows, width, dtype, x, n_src, rows, row_div, codes, scales,
                          stream=None):
    st, dev = _where(stream)
    kb = (width + 127) // 128
    _check(_lib.moelora_quantize_rows(
        n_rows, width, dtype, _buf(x, n_src * width, _dt(dtype), dev, "x"), n_src,
        _buf(rows, n_rows, _INT, dev, "rows", True), row_div,
        _buf(codes, n_rows * kb * 128, _BYTE, dev, "codes"),
        _buf(scales, n_rows * kb, _FLT, dev, "scales"), st), "moelora_quantize_rows")


def moelora_quantize_weights(n_mats, rows, width, dtype, w, codes, scales, codes_t=None,
                             scales_t=None, stream=None):
    st, dev = _where(stream)
    kb, nb = (width + 127) // 128, (rows + 127) // 128
    _check(_lib.moelora_quantize_weights(
        n_mats, rows, width, dtype, _buf(w, n_mats * rows * width, _dt(dtype), dev, "w"),
        _buf(codes, n_mats * rows * kb * 128, _BYTE, dev, "codes"),
        _buf(scales, n_mats * nb * kb, _FLT, dev, "scales"),
        _buf(codes_t, n_mats * width * nb * 128, _BYTE, dev, "codes_t", True),
        _buf(scales_t, n_mats * nb * kb, _FLT, dev, "scales_t", True), st),
        "moelora_quantize_weights")


def moelora_fp8_gemm(n_rows, n_out, width, n_experts, out_dtype, flags, codes, scales,
                     expert_start, w_codes, w_scales, out, stream=None):
    st, dev = _where(stream)
    kb, nb = (width + 127) // 128, (n_out + 127) // 128
    mats = n_experts * (2 if flags & FP8_SILU_MUL else 1)
    _check(_lib.moelora_fp8_gemm(
        n_rows, n_out, width, n_experts, out_dtype, flags,
        _buf(codes, n_rows * kb * 128, _BYTE, dev, "codes"), _buf(scales, n_rows * kb, _FLT, dev, "scales"),
        _buf(expert_start, n_experts + 1, _INT, dev, "expert_start", True),
        _buf(w_codes, mats * n_out * kb * 128, _BYTE, dev, "w_codes"),
        _buf(w_scales, mats * nb * kb, _FLT, dev, "w_scales"),
        _buf(out, n_rows * n_out, _dt(out_dtype), dev, "out"), st), "moelora_fp8_gemm")


def moelora_fp8_gemm_info(n_rows, n_out, width, n_experts, out_dtype, flags=0):
    """-> one line on the kernel that such a product takes."""
    buf = ctypes.create_string_buffer(128)
    _check(_lib.moelora_fp8_gemm_info(n_rows, n_out, width, n_experts, out_dtype, flags, buf, len(buf)),
           "moelora_fp8_gemm_info")
    return buf.value.decode()


class Plan:
    """Owning wrapper of a plan handle."""

    _destroy_fn = _lib.moelora_plan_destroy  # ctypes function object (holds the library)

    def __init__(self, max_tokens, hidden, inter, n_experts, top_k, n_adapters, rank,
                 dtype, flags=0):
        self.handle, self.workspace_bytes = moelora_plan(
            max_tokens, hidden, inter, n_experts, top_k, n_adapters, rank, dtype, flags)
        self.desc = dict(max_tokens=max_tokens, hidden=hidden, inter=inter,
                         n_experts=n_experts, top_k=top_k, n_adapters=n_adapters,
                         rank=rank, dtype=dtype)

    def __del__(self):
        # the destroy function is held by the class: module globals may
        # already be gone when a plan is collected at interpreter shutdown
        h = getattr(self, "handle", None)
        if h:
            self._destroy_fn(h)
            self.handle = None

    def layout(self, n_tokens):
        return moelora_workspace_layout(self.handle, n_tokens)

    def info(self, n_tokens):
        return moelora_plan_info(self.handle, n_tokens)

    def forward(self, n_tokens, x, out, workspace, *, router_logits=None, topk_ids=None,
                topk_w=None, adapter_ids=None, w_gate_up, w_down, lora_a_gu=None,
                lora_b_gu=None, lora_a_d=None, lora_b_d=None, stream=None):
        ws_bytes = workspace.numel() * workspace.element_size() \
            if hasattr(workspace, "numel") else self.workspace_bytes
        moelora_forward(self.handle, n_tokens, x, router_logits, topk_ids, topk_w,
                        adapter_ids, w_gate_up, w_down, lora_a_gu, lora_b_gu, lora_a_d,
                        lora_b_d, out, workspace, ws_bytes, stream)
