"""Every kernel that a product on 4-bit weights can take, on random data of several
uneven and empty experts, with contractions that end inside a slab and inside 16
bytes.  Which kernel a case takes is asserted on the host, so a changed rule
cannot quietly leave one without a case.

Beside the bound for each element, the norm of all errors is held to what normal
data give: some K / 32 + 16 float32 roundings of partial sums no larger than the
result, at random or all one way: under (K / 32 + 16) 2^-23 of the norm (three times as
many for float32 rows), plus the last rounding, 2^-8 for bf16, whose mean square is
a third of its largest; SiLU multiplies the former by at most 2.1.  One product too many or
too few of K = 5000 is 1e-2 of a typical result, one bit of a scale far more."""
import numpy as np
import pytest
import torch

from test_fp4 import DT, check, lib, make, product64, say

ROWS = {
    "few": [2, 0, 5, 1, 0, 0, 3, 16, 17, 1, 0],
    "many_few": [2, 1, 0, 5, 3, 1, 0, 9] * 8,
    "little": [17, 0, 33, 64, 1, 30],
    "mid": [25, 40, 0, 64, 65, 7],
    "eighty": [130, 0, 90, 127, 1, 57, 200, 129],
    "hundreds": [130, 0, 300, 127, 1, 257, 400],
    "one": [1],
    "three": [3],
    "forty": [40],
    "skew": [0] * 30 + [90] + [1] * 3,
}
F, B = lib.F32, lib.BF16
# kernel, row types, SiLU, rows, columns, contractions
CASES = [
    ("short", (F, B), 0, "mid", 300, (1, 3)),
    ("short", (F, B), 1, "mid", 300, (2, 3)),
    ("short", (B,), 0, "skew", 40, (7,)),
    ("stream2", (F, B), 0, "few", 70, (384, 1003, 5000)),
    ("stream2", (F, B), 1, "few", 70, (384, 1003, 5000)),
    ("stream2", (F, B), 0, "one", 2000, (8, 700)),
    ("stream2", (F, B), 1, "three", 999, (1500,)),
    ("stream2", (F, B), 0, "skew", 40, (520,)),
    ("stream4_once", (B,), 0, "many_few", 520, (384, 1003)),
    ("stream4_once", (B,), 1, "many_few", 270, (384, 1003, 2600)),
    ("split1x1", (F, B), 0, "little", 70, (384, 1003, 5000)),
    ("split1x1", (F, B), 1, "little", 70, (384, 1003, 5000)),
    ("split1x1", (F, B), 0, "forty", 1, (100, 1500)),
    ("split2x2", (B,), 0, "mid", 2600, (384, 1003, 5000)),
    ("split2x2", (B,), 1, "mid", 1500, (384, 1003, 5000)),
    ("split2x2", (F,), 0, "mid", 1900, (384, 1003, 5000)),
    ("split2x2", (F,), 1, "mid", 1300, (384, 1003, 5000)),
    ("tile4x1", (F,), 0, "mid", 4100, (384, 1003)),
    ("tile4x1", (F,), 1, "mid", 2050, (384, 1003, 2600)),
    ("tile4x1", (F,), 0, "many_few", 520, (1003,)),
    ("tile4x2", (F,), 0, "hundreds", 4100, (384, 1003)),
    ("tile4x2", (F,), 1, "hundreds", 2050, (384, 1003)),
    ("tile4x2", (B,), 0, "hundreds", 1500, (385, 1003)),
    ("tile4x2", (B,), 1, "eighty", 1500, (385, 1003)),
    ("tile2x2", (B,), 0, "hundreds", 1500, (384, 1000, 2600)),
    ("tile2x2", (B,), 1, "eighty", 1500, (384, 1000, 2600)),
    ("tile4x2_once", (B,), 0, "mid", 8100, (384, 1003)),
    ("tile4x2_once", (B,), 1, "mid", 4100, (384, 1003, 2600)),
    ("tile4x4", (B,), 0, "hundreds", 9001, (384, 1000)),
    ("tile4x4", (B,), 1, "hundreds", 4100, (384, 1000, 5000)),
    ("tile4x4_regs", (B,), 0, "hundreds", 9001, (385, 1003)),
    ("tile4x4_regs", (B,), 1, "hundreds", 4100, (385, 1003, 5001)),
]
FLAT = [(k, t, s, r, n, c) for k, ts, s, r, n, cs in CASES for t in ts for c in cs]


def kernel(rows, N, K, dtype, silu):
    line = lib.moelora_fp4_gemm_info(sum(ROWS[rows]), N, K, len(ROWS[rows]), dtype, silu)
    return dict(p.split("=") for p in line.split())["kernel"]


def test_each_case_takes_its_kernel():
    for name, dtype, silu, rows, N, K in FLAT:
        assert kernel(rows, N, K, dtype, silu) == name, (rows, N, K, dtype, silu)
    common = {"short", "stream2", "split1x1", "split2x2", "tile4x2"}
    for dtype, own in ((F, {"tile4x1"}), (B, {"stream4_once", "tile2x2", "tile4x2_once", "tile4x4", "tile4x4_regs"})):
        for silu in (0, 1):
            assert {c[0] for c in FLAT if c[1] == dtype and c[2] == silu} == common | own


def test_workgroups_of_short_rows_are_bounded():
    """Workgroups of 256 threads for 256 columns, an expert and every so many rows: no more than 2^30
    threads at the limits, no third dimension past its own."""
    for R, N, E in ((1 << 17, 131072, 1024), (1 << 24, 1024, 1), (1 << 24, 1, 1024), (1, 1, 1), (5, 131072, 1024)):
        line = dict(p.split("=") for p in lib.moelora_fp4_gemm_info(R, N, 3, E, B).split())
        groups, columns = int(line["groups"]), (N + 255) // 256
        assert line["kernel"] == "short" and 1 <= groups <= 256 and groups * columns * min(E, R) * 256 <= 1 << 30


def test_info_refuses():
    assert lib.moelora_fp4_gemm_info(0, 8, 8, 1, F) == "kernel=none"
    for bad in ((-1, 8, 8, 1, F), (4, 0, 8, 1, F), (4, 8, 8, 1025, F), (4, 8, 8, 1, 2), (4, 8, 8, 1, F, 2)):
        with pytest.raises(lib.MoeLoraError):
            lib.moelora_fp4_gemm_info(*bad)


@pytest.mark.gpu
@pytest.mark.parametrize("name,dtype,silu,rows,N,K", FLAT)
def test_kernel(name, dtype, silu, rows, N, K):
    cs = ROWS[rows]
    R, gap = sum(cs), 3
    say(f"[fp4] {name} {rows} N={N} K={K} silu={silu} {DT[dtype]}")
    x, tc, ts, w, start = make(cs, N, K, 2 if silu else 1, dtype, N + K, gap)
    x[R:] = float("nan")
    buf = torch.full((R + gap + 64, N), -7.0, dtype=DT[dtype], device="cuda")
    out = buf[32:32 + R + gap] if 64 * N % 16 == 0 else buf[16 * 2:16 * 2 + R + gap]
    lib.moelora_fp4_gemm(R + gap, N, K, len(cs), dtype, silu, x, start, tc, ts, out)
    ref, err = product64(x[:R], w, cs, silu)
    check(out[:R], ref, err)
    assert bool((buf[:32] == -7).all()) and bool((buf[32 + R:] == -7).all())
    sums = (K / 32 + 16) * 2.0 ** -23 * (3 if dtype == F else 1) * (2.1 if silu else 1)
    half = 2.0 ** -24 if dtype == F else 2.0 ** -9
    far = float((out[:R].double() - ref).norm() / ref.norm())
    assert far <= sums + 1.2 * half, far


@pytest.mark.gpu
@pytest.mark.parametrize("K", [8, 9, 15, 16, 127, 128, 129, 136, 255, 257, 511, 512, 513, 640])
def test_ends_of_rows(K):
    """Rows that end anywhere in a slab, beside rows of NaN: nothing past an end
    gets in, through every way the rows are loaded."""
    for dtype in (F, B):
        for counts, N in (([3], 40), ([30, 0, 41], 70), ([50, 60], 2100), ([130, 90, 300], 4100)):
            R = sum(counts)
            x, tc, ts, w, start = make(counts, N, K, 1, dtype, K, 2)
            x[R:] = float("nan")
            x[R - 1] = float("inf")
            out = torch.zeros(R + 2, N, dtype=DT[dtype], device="cuda")
            lib.moelora_fp4_gemm(R + 2, N, K, len(counts), dtype, 0, x, start, tc, ts, out)
            ref, err = product64(x[:R - 1], w, counts[:-1] + [counts[-1] - 1], 0)
            check(out[:R - 1], ref, err)
