"""Infinities in the rows of the product on 4-bit weights: results are what the formula gives,
an infinity, or NaN where it meets a zero weight or one of the other sign, for both types of rows
and through every kernel of float32 rows; the other rows are to the bit what they are without."""
import pytest
import torch

from test_fp4 import DT, lib, make, say
from test_fp4_kernels import FLAT, ROWS, kernel

pytestmark = pytest.mark.gpu
F, B = lib.F32, lib.BF16
INF, NAN = float("inf"), float("nan")
FIRST = {}
for name, dtype, silu, rows, N, K in FLAT:
    FIRST.setdefault((name, dtype, silu), (rows, N, K))
CASES = [(*k, *v) for k, v in FIRST.items() if k[1] == F or k[0] in ("stream2", "tile4x4")]


def formula(x, w, silu):
    """One row, float64: sums of products term by term."""
    y = [(x.double()[None] * m).sum(1) for m in w]
    return y[0] * torch.sigmoid(y[0]) * y[1] if silu else y[0]


@pytest.mark.parametrize("name,dtype,silu,rows,N,K", CASES)
def test_infinite_elements(name, dtype, silu, rows, N, K):
    say(f"[fp4] infinities {name} {rows} N={N} K={K} silu={silu} {DT[dtype]}")
    assert kernel(rows, N, K, dtype, silu) == name
    cs, halves = ROWS[rows], 2 if silu else 1
    R = sum(cs)
    x, tc, ts, w, start = make(cs, N, K, halves, dtype, N + K)
    expert = torch.repeat_interleave(torch.arange(len(cs)), torch.tensor(cs))
    clean, out = (torch.zeros(R, N, dtype=DT[dtype], device="cuda") for _ in range(2))
    lib.moelora_fp4_gemm(R, N, K, len(cs), dtype, silu, x, start, tc, ts, clean)
    assert bool(torch.isfinite(clean).all())
    odd = sorted({0, R // 2, R - 1})
    for put in ({0: INF}, {K - 1: -INF}, {K // 2: INF, K - 1: INF}, {0: -INF, K - 1: NAN}):
        y = x.clone()
        for r in odd:
            for k, v in put.items():
                y[r, k] = v
        lib.moelora_fp4_gemm(R, N, K, len(cs), dtype, silu, y, start, tc, ts, out)
        for r in odd:
            e = int(expert[r])
            want, got = formula(y[r], w[e * halves:(e + 1) * halves], silu), out[r].double()
            assert torch.equal(got.isnan(), want.isnan())
            assert torch.equal(got.nan_to_num(0, 1, -1), want.nan_to_num(0, 1, -1))
        rest = torch.tensor([r not in odd for r in range(R)], device="cuda")
        assert torch.equal(out[rest], clean[rest])


def test_a_nan_is_no_infinity():
    """NaN whose upper half alone would read as an infinity, beside an infinity."""
    for R in (1, 40):
        x, tc, ts, w, start = make([R], 96, 300, 1, F, 3)
        x.view(torch.int32)[0, 7] = 0x7f800001
        x[0, 6] = INF
        out = torch.zeros(R, 96, device="cuda")
        lib.moelora_fp4_gemm(R, 96, 300, 1, F, 0, x, start, tc, ts, out)
        assert bool(out[0].isnan().all()) and bool(torch.isfinite(out[1:]).all())
