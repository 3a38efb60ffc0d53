"""Argument checks of the stand-alone operators (no GPU needed): every call
here is refused on the host, before any device is touched."""
import ctypes

import pytest
import torch

lib = pytest.importorskip("lora_expert_gemm_amd")

A = 4096          # an aligned address that no call here may read
B = A + 8         # 8-byte aligned only
OK = lib.OK
S = 0             # the null stream


def status(fn, *args):
    return getattr(lib._lib, fn)(*args)


def dispatch(T=4, H=8, E=4, k=2, dtype=lib.F32, x=A, ids=A, start=A, rows=A, pos=A, xs=A, ws=A,
             ws_bytes=1 << 20):
    return status("moelora_dispatch", T, H, E, k, dtype, x, ids, start, rows, pos, xs, ws,
                  ws_bytes, S)


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), lib.ERR_INVALID_ARG),
    (dict(H=0), lib.ERR_UNSUPPORTED),
    (dict(H=65537), lib.ERR_UNSUPPORTED),
    (dict(E=0), lib.ERR_UNSUPPORTED),
    (dict(E=1025), lib.ERR_UNSUPPORTED),
    (dict(k=0), lib.ERR_UNSUPPORTED),
    (dict(k=33), lib.ERR_UNSUPPORTED),
    (dict(T=(1 << 24) + 1, k=1), lib.ERR_UNSUPPORTED),
    (dict(T=1 << 23, k=3), lib.ERR_UNSUPPORTED),
    (dict(dtype=lib.BF16_FP8W), lib.ERR_UNSUPPORTED),
    (dict(dtype=-1), lib.ERR_UNSUPPORTED),
    (dict(start=None), lib.ERR_INVALID_ARG),
    (dict(start=None, T=0), lib.ERR_INVALID_ARG),
    (dict(ids=None), lib.ERR_INVALID_ARG),
    (dict(rows=None), lib.ERR_INVALID_ARG),
    (dict(pos=None), lib.ERR_INVALID_ARG),
    (dict(x=None), lib.ERR_INVALID_ARG),       # xs without x
    (dict(x=B), lib.ERR_INVALID_ARG),
    (dict(ids=B), lib.ERR_INVALID_ARG),
    (dict(pos=B), lib.ERR_INVALID_ARG),
    (dict(xs=B), lib.ERR_INVALID_ARG),
    (dict(T=1 << 20, ws=None), lib.ERR_INVALID_ARG),
    (dict(T=1 << 20, ws_bytes=64), lib.ERR_WORKSPACE),
])
def test_dispatch_refuses(bad, want):
    assert dispatch(**bad) == want


def test_dispatch_workspace():
    assert lib.moelora_dispatch_workspace(0, 4, 2) == 0
    assert lib.moelora_dispatch_workspace(16, 1024, 4) == 0
    for T, k, E in ((1 << 24, 1, 1024), (1 << 19, 32, 7), (6400, 4, 32), (100_003, 8, 128)):
        n = lib.moelora_dispatch_workspace(T, E, k)
        assert 0 < n <= 1024 * E
    with pytest.raises(lib.MoeLoraError) as ei:
        lib.moelora_dispatch_workspace(4, 1025, 2)
    assert ei.value.status == lib.ERR_UNSUPPORTED
    assert status("moelora_dispatch_workspace", 4, 4, 2, None) == lib.ERR_INVALID_ARG


@pytest.mark.parametrize("args,want", [
    ((-1, 8, 2, lib.F32, A, A, A, S), lib.ERR_INVALID_ARG),
    ((4, 8, 2, 9, A, A, A, S), lib.ERR_UNSUPPORTED),
    ((4, 8, 2, lib.F32, None, A, A, S), lib.ERR_INVALID_ARG),
    ((4, 8, 2, lib.F32, A, None, A, S), lib.ERR_INVALID_ARG),
    ((4, 8, 2, lib.F32, A, A, B, S), lib.ERR_INVALID_ARG),
    ((0, 8, 2, lib.F32, None, None, None, S), OK),
])
def test_dispatch_backward_refuses(args, want):
    assert status("moelora_dispatch_backward", *args) == want


@pytest.mark.parametrize("args,want", [
    ((4, 8, 33, lib.F32, A, A, A, A, S), lib.ERR_UNSUPPORTED),
    ((4, 8, 2, lib.F32, A, A, None, A, S), lib.ERR_INVALID_ARG),   # weights are required
    ((4, 8, 2, lib.F32, B, A, A, A, S), lib.ERR_INVALID_ARG),
    ((0, 8, 2, lib.F32, None, None, None, None, S), OK),
])
def test_combine_refuses(args, want):
    assert status("moelora_combine", *args) == want


@pytest.mark.parametrize("args,want", [
    # dout, ys, row_pos, topk_w, dys, dw
    ((A, A, A, A, None, None), lib.ERR_INVALID_ARG),   # nothing wanted
    ((A, None, A, A, A, A), lib.ERR_INVALID_ARG),      # dw needs ys
    ((A, A, A, None, A, A), lib.ERR_INVALID_ARG),      # dys needs the weights
    ((None, A, A, A, A, A), lib.ERR_INVALID_ARG),
    ((A, A, None, A, A, A), lib.ERR_INVALID_ARG),
    ((A, A, A, A, B, A), lib.ERR_INVALID_ARG),
    ((A, A, A, A, A, B), lib.ERR_INVALID_ARG),
])
def test_combine_backward_refuses(args, want):
    assert status("moelora_combine_backward", 4, 8, 2, lib.F32, *args, S) == want


def rows(n=4, width=8, dtype=lib.F32, x=A, n_src=4, index=None, div=1, codes=A, scales=A):
    return status("moelora_quantize_rows", n, width, dtype, x, n_src, index, div, codes, scales, S)


@pytest.mark.parametrize("bad,want", [
    (dict(n=-1), lib.ERR_INVALID_ARG),
    (dict(n_src=-1), lib.ERR_INVALID_ARG),
    (dict(n_src=3), lib.ERR_INVALID_ARG),              # no index: rows 0 .. n-1 of x
    (dict(div=2), lib.ERR_INVALID_ARG),
    (dict(index=A, div=0), lib.ERR_INVALID_ARG),
    (dict(width=0), lib.ERR_UNSUPPORTED),
    (dict(width=65537), lib.ERR_UNSUPPORTED),
    (dict(n=(1 << 24) + 1, n_src=(1 << 24) + 1), lib.ERR_UNSUPPORTED),
    (dict(dtype=2), lib.ERR_UNSUPPORTED),
    (dict(x=None), lib.ERR_INVALID_ARG),
    (dict(codes=B), lib.ERR_INVALID_ARG),
    (dict(scales=None), lib.ERR_INVALID_ARG),
    (dict(index=B), lib.ERR_INVALID_ARG),
    (dict(n=0, x=None, codes=None, scales=None), OK),
])
def test_quantize_rows_refuses(bad, want):
    assert rows(**bad) == want


@pytest.mark.parametrize("args,want", [
    ((-1, 8, 8, lib.F32, A, A, A, None, None), lib.ERR_INVALID_ARG),
    ((65536, 8, 8, lib.F32, A, A, A, None, None), lib.ERR_UNSUPPORTED),
    ((1, 131073, 8, lib.F32, A, A, A, None, None), lib.ERR_UNSUPPORTED),
    ((1, 8, 0, lib.F32, A, A, A, None, None), lib.ERR_UNSUPPORTED),
    ((1, 8, 8, 5, A, A, A, None, None), lib.ERR_UNSUPPORTED),
    ((1, 8, 8, lib.F32, A, A, A, A, None), lib.ERR_INVALID_ARG),   # both or neither
    ((1, 8, 8, lib.F32, A, A, A, None, A), lib.ERR_INVALID_ARG),
    ((1, 8, 8, lib.F32, B, A, A, None, None), lib.ERR_INVALID_ARG),
    ((0, 8, 8, lib.F32, None, None, None, None, None), OK),
])
def test_quantize_weights_refuses(args, want):
    assert status("moelora_quantize_weights", *args, S) == want


def gemm(M=4, N=8, K=8, E=1, out_dtype=lib.F32, flags=0, codes=A, scales=A, start=None, w=A, ws=A,
         out=A):
    return status("moelora_fp8_gemm", M, N, K, E, out_dtype, flags, codes, scales, start, w, ws,
                  out, S)


@pytest.mark.parametrize("bad,want", [
    (dict(M=-1), lib.ERR_INVALID_ARG),
    (dict(M=(1 << 24) + 1), lib.ERR_UNSUPPORTED),
    (dict(N=0), lib.ERR_UNSUPPORTED),
    (dict(N=131073), lib.ERR_UNSUPPORTED),
    (dict(K=0), lib.ERR_UNSUPPORTED),
    (dict(K=65537), lib.ERR_UNSUPPORTED),
    (dict(E=0), lib.ERR_UNSUPPORTED),
    (dict(E=1025, start=A), lib.ERR_UNSUPPORTED),
    (dict(E=2), lib.ERR_INVALID_ARG),                 # several experts need their ranges
    (dict(flags=2), lib.ERR_UNSUPPORTED),
    (dict(out_dtype=2), lib.ERR_UNSUPPORTED),
    (dict(codes=None), lib.ERR_INVALID_ARG),
    (dict(scales=B), lib.ERR_INVALID_ARG),
    (dict(start=B), lib.ERR_INVALID_ARG),
    (dict(w=B), lib.ERR_INVALID_ARG),
    (dict(ws=None), lib.ERR_INVALID_ARG),
    (dict(out=B), lib.ERR_INVALID_ARG),
    (dict(M=0, codes=None, scales=None, w=None, ws=None, out=None), OK),
])
def test_fp8_gemm_refuses(bad, want):
    assert gemm(**bad) == want


def test_tensor_arguments_are_checked():
    """The binding refuses tensors that are too small, of another element
    size, strided, or not on the current device."""
    x = torch.zeros(4, 8)
    for bad in (x[:2], x.double(), x.t(), x):   # the last: on the CPU
        with pytest.raises(ValueError):
            lib.moelora_combine(4, 8, 1, lib.F32, bad, A, A, A, stream=0)
    with pytest.raises(ValueError):
        lib.moelora_combine(4, 8, 1, lib.F32, None, A, A, A, stream=0)


def test_tensors_of_another_type_are_refused():
    """The same bytes an element are not enough: float16 rows read as bfloat16
    would be silently wrong."""
    f32, f16, i32 = torch.zeros(64), torch.zeros(64, dtype=torch.float16), torch.zeros(64, dtype=torch.int32)
    wrong = "expected a contiguous tensor"
    for call in (
            lambda: lib.moelora_combine(4, 8, 1, lib.BF16, f16, A, A, A, stream=0),
            lambda: lib.moelora_combine(4, 8, 1, lib.F32, i32, A, A, A, stream=0),
            lambda: lib.moelora_combine(4, 8, 1, lib.F32, A, f32, A, A, stream=0),
            lambda: lib.moelora_combine(4, 8, 1, lib.F32, A, A, i32, A, stream=0),
            lambda: lib.moelora_dispatch(4, 8, 4, 2, lib.F32, A, f32, A, A, A, A, A, 64, stream=0),
            lambda: lib.moelora_dispatch_backward(4, 8, 2, lib.BF16, f16, A, A, stream=0),
            lambda: lib.moelora_quantize_rows(4, 8, lib.BF16, f16, 4, None, 1, A, A, stream=0),
            lambda: lib.moelora_quantize_rows(4, 8, lib.BF16, A, 4, None, 1, f32, A, stream=0),
            lambda: lib.moelora_quantize_weights(1, 4, 8, lib.BF16, f16, A, A, stream=0),
            lambda: lib.moelora_fp8_gemm(4, 8, 8, 1, lib.BF16, 0, A, A, f32, A, A, A, stream=0),
            lambda: lib.moelora_fp8_gemm(4, 8, 8, 1, lib.BF16, 0, A, A, None, A, A, f16, stream=0)):
        with pytest.raises(ValueError, match=wrong):
            call()


def test_a_stream_of_another_device_is_refused(monkeypatch):
    class Stream:
        device_index, cuda_stream = 1, 0
    monkeypatch.setattr(torch, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="stream is on device 1"):
        lib.moelora_combine(4, 8, 1, lib.F32, A, A, A, A, stream=Stream())


def test_entry_points_have_bindings():
    for n in lib.exported_symbols():
        assert hasattr(lib, n), n
        assert isinstance(getattr(lib._lib, n), ctypes._CFuncPtr)
