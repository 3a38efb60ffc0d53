"""Argument checks of the router's operators and of the 4-bit weights and their
product (no GPU needed): every call here is refused on the host, before any
device is touched."""
import pytest
import torch

lib = pytest.importorskip("lora_expert_gemm_amd")

A = 4096          # an aligned address that no call here may read
B = A + 8         # 8-byte aligned only
OK, BAD, NOT = lib.OK, lib.ERR_INVALID_ARG, lib.ERR_UNSUPPORTED
S = 0             # the null stream


def status(fn, *args):
    return getattr(lib._lib, fn)(*args)


SHAPES = [
    (dict(T=-1), BAD),
    (dict(E=0), NOT),
    (dict(E=1025), NOT),
    (dict(k=0), NOT),
    (dict(k=33, E=64), NOT),
    (dict(k=5, E=4), NOT),                       # more picks than experts
    (dict(T=(1 << 24) + 1, k=1), NOT),
    (dict(T=1 << 23, k=3), NOT),
    (dict(dtype=2), NOT),
    (dict(dtype=-1), NOT),
    (dict(logits=None), BAD),
    (dict(logits=B), BAD),
    (dict(mask=B), BAD),
]


def route(T=4, E=4, k=2, dtype=lib.F32, flags=0, logits=A, mask=None, ids=A, w=A):
    return status("moelora_route", T, E, k, dtype, flags, logits, mask, ids, w, S)


@pytest.mark.parametrize("bad,want", SHAPES + [
    (dict(flags=2), NOT),
    (dict(ids=None), BAD),
    (dict(w=B), BAD),
    (dict(T=0, logits=None, ids=None, w=None), OK),
    (dict(T=0, flags=4), NOT),
])
def test_route_refuses(bad, want):
    assert route(**bad) == want


def balance(T=4, E=4, k=2, dtype=lib.F32, logits=A, mask=None, ids=A, counts=A, sums=A, loss=A, ws=A,
            ws_bytes=1 << 24):
    return status("moelora_balance_loss", T, E, k, dtype, logits, mask, ids, counts, sums, loss, ws, ws_bytes, S)


@pytest.mark.parametrize("bad,want", SHAPES + [
    (dict(ids=None), BAD),
    (dict(counts=None), BAD),
    (dict(counts=None, T=0), BAD),
    (dict(sums=B), BAD),
    (dict(loss=None), BAD),
    (dict(T=1 << 20, ws=None), BAD),
    (dict(T=1 << 20, ws=B), BAD),
    (dict(T=1 << 20, ws_bytes=64), lib.ERR_WORKSPACE),
])
def test_balance_refuses(bad, want):
    assert balance(**bad) == want


def test_balance_workspace():
    assert lib.moelora_balance_loss_workspace(0, 4, 2) == 0
    assert lib.moelora_balance_loss_workspace(16, 1024, 4) == 0
    for E in (1, 2, 7, 32, 129, 1024):
        sizes = [lib.moelora_balance_loss_workspace(T, E, 1) for T in
                 (0, 1, 31, 32, 33, 100, 1000, 4096, 4097, 8191, 8192, 8193, 32768, 32769, 100_003, 1 << 24)]
        assert sizes == sorted(sizes)          # one for the largest batch serves the smaller ones
        assert 0 < sizes[-1] <= 4096 * (E + 2)
    with pytest.raises(lib.MoeLoraError) as ei:
        lib.moelora_balance_loss_workspace(4, 1025, 2)
    assert ei.value.status == NOT
    assert status("moelora_balance_loss_workspace", 4, 4, 2, None) == BAD


def backward(T=4, E=4, k=2, dtype=lib.F32, flags=0, logits=A, mask=None, ids=A, w=A, dw=A, counts=A, dloss=A,
             dlogits=A):
    return status("moelora_route_backward", T, E, k, dtype, flags, logits, mask, ids, w, dw, counts, dloss,
                  dlogits, S)


@pytest.mark.parametrize("bad,want", SHAPES + [
    (dict(flags=2), NOT),
    (dict(dlogits=None), BAD),
    (dict(dlogits=B), BAD),
    (dict(dw=None, counts=None, dloss=None), BAD),   # nothing wanted
    (dict(counts=None), BAD),                        # dloss needs the counts
    (dict(dloss=None), BAD),
    (dict(ids=None), BAD),
    (dict(w=None), BAD),
    (dict(w=B, dw=None), BAD),
    (dict(T=0, logits=None, dlogits=None), OK),
])
def test_backward_refuses(bad, want):
    assert backward(**bad) == want


SIZES = [
    (dict(mats=-1), BAD),
    (dict(mats=65536), NOT),
    (dict(N=0), NOT),
    (dict(N=131073), NOT),
    (dict(K=0), NOT),
    (dict(K=65537), NOT),
    (dict(mats=65535, N=131072, K=65536), NOT),      # more than a launch holds
    (dict(mats=64, N=131072, K=65536), NOT),
    (dict(mats=0, src=None, codes=None, scales=None), OK),
    (dict(src=None), BAD),
    (dict(codes=B), BAD),
    (dict(scales=None), BAD),
]


@pytest.mark.parametrize("bad,want", SIZES + [(dict(dtype=2), NOT), (dict(dtype=3, mats=0), NOT)])
def test_quantize_and_dequantize_refuse(bad, want):
    def call(fn, mats=1, N=8, K=8, dtype=lib.F32, src=A, codes=A, scales=A):
        w = (src, codes, scales) if fn == "quantize" else (codes, scales, src)
        return status(f"moelora_{fn}_weights_fp4", mats, N, K, dtype, *w, S)
    assert call("quantize", **bad) == want
    assert call("dequantize", **bad) == want


@pytest.mark.parametrize("bad,want", SIZES + [(dict(given=None), BAD), (dict(given=B), BAD)])
def test_pack_refuses(bad, want):
    def call(mats=1, N=8, K=8, src=A, given=A, codes=A, scales=A):
        return status("moelora_pack_weights_fp4", mats, N, K, src, given, codes, scales, S)
    assert call(**bad) == want


def gemm(M=4, N=8, K=8, E=1, dtype=lib.F32, flags=0, x=A, start=None, w=A, ws=A, out=A):
    return status("moelora_fp4_gemm", M, N, K, E, dtype, flags, x, start, w, ws, out, S)


@pytest.mark.parametrize("bad,want", [
    (dict(M=-1), BAD),
    (dict(M=(1 << 24) + 1), NOT),
    (dict(M=(1 << 24) - 1, N=1026), NOT),            # more results than a launch makes
    (dict(N=0), NOT),
    (dict(N=131073), NOT),
    (dict(K=0), NOT),
    (dict(K=65537), NOT),
    (dict(E=0), NOT),
    (dict(E=1025, start=A), NOT),
    (dict(E=1024, start=A, N=131072, K=65536), NOT),
    (dict(E=2), BAD),                                # several experts need their ranges
    (dict(flags=2), NOT),
    (dict(dtype=2), NOT),
    (dict(x=None), BAD),
    (dict(start=B), BAD),
    (dict(w=B), BAD),
    (dict(ws=None), BAD),
    (dict(out=B), BAD),
    (dict(M=0, x=None, w=None, ws=None, out=None), OK),
])
def test_fp4_gemm_refuses(bad, want):
    assert gemm(**bad) == want


def test_tensors_are_checked():
    """Too small, of another type, strided, or not on the current device."""
    f32, f16 = torch.zeros(4, 16), torch.zeros(4, 16, dtype=torch.float16)
    i32, u8 = torch.zeros(64, dtype=torch.int32), torch.zeros(4096, dtype=torch.uint8)
    for bad in (f32[:3], f32.t(), f16, f32):       # the last: on the CPU
        for call in (
                lambda: lib.moelora_route(4, 16, 2, lib.F32, 0, bad, None, A, A, stream=0),
                lambda: lib.moelora_balance_loss(4, 16, 2, lib.F32, bad, None, A, A, A, A, None, 0, stream=0),
                lambda: lib.moelora_route_backward(4, 16, 2, lib.F32, 0, A, None, A, A, A, A, A, bad, stream=0),
                lambda: lib.moelora_quantize_weights_fp4(1, 4, 16, lib.F32, bad, A, A, stream=0),
                lambda: lib.moelora_dequantize_weights_fp4(1, 4, 16, lib.F32, A, A, bad, stream=0),
                lambda: lib.moelora_fp4_gemm(4, 8, 16, 1, lib.F32, 0, bad, None, A, A, A, stream=0)):
            with pytest.raises(ValueError):
                call()
    wrong = "expected a contiguous tensor"
    for call in (
            lambda: lib.moelora_route(4, 16, 2, lib.F32, 0, A, i32, A, A, stream=0),         # mask: bytes
            lambda: lib.moelora_route(4, 16, 2, lib.F32, 0, A, None, f32, A, stream=0),
            lambda: lib.moelora_route(4, 16, 2, lib.F32, 0, A, None, A, i32, stream=0),
            lambda: lib.moelora_balance_loss(4, 16, 2, lib.F32, A, None, A, i32[:16], A, A, None, 0, stream=0),
            lambda: lib.moelora_balance_loss(4, 16, 2, lib.F32, A, None, A, A, A, f32[0, :1], None, 0, stream=0),
            lambda: lib.moelora_balance_loss(4, 16, 2, lib.F32, A, None, A, A, A, A, u8, 5000, stream=0),
            lambda: lib.moelora_route_backward(4, 16, 2, lib.F32, 0, A, None, A, A, f32[0, :7], A, A, A, stream=0),
            lambda: lib.moelora_quantize_weights_fp4(1, 17, 16, lib.F32, A, u8[:2047], A, stream=0),
            lambda: lib.moelora_quantize_weights_fp4(1, 17, 16, lib.F32, A, A, u8[:511], stream=0),
            lambda: lib.moelora_pack_weights_fp4(1, 4, 33, u8[:67], A, A, A, stream=0),
            lambda: lib.moelora_pack_weights_fp4(1, 4, 33, A, u8[:7], A, A, stream=0),
            lambda: lib.moelora_dequantize_weights_fp4(1, 16, 129, lib.F32, u8[:2047], A, A, stream=0),
            lambda: lib.moelora_fp4_gemm(4, 16, 16, 1, lib.F32, 1, A, None, u8[:2047], A, A, stream=0),
            lambda: lib.moelora_fp4_gemm(4, 16, 16, 1, lib.F32, 0, A, None, A, A, f32[:3], stream=0)):
        with pytest.raises(ValueError, match=wrong):
            call()
