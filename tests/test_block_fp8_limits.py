"""The block-scaled product at the ends of its range, against 64 bits.

Scales: any two finite float32 scales of a block, also where their product is
no normal float32 though the scaled block sum is.  One that overflows is exact
all the same.  One below 2^-126 is a multiple of 2^-149, off by at most 2^-150,
and meets a block sum of at most 128 448^2 < 2^25: its block is off by less than
2^-125."""
import math

import pytest
import torch

from test_block_fp8 import DT, TABLE, check, lib, make, product64, say, up

pytestmark = pytest.mark.gpu

# rows of each expert, columns: the streamed kernel with one and two row groups
# a workgroup, short rows an expert in tiles, tiles of 32, 64 and 128 rows
SCALED = [([4], 40), ([30], 40), ([3, 0, 5], 40), ([2] * 64, 2880), ([40, 0, 33], 200), ([300], 900),
          ([90, 70, 0, 110], 3000), ([900], 9000), ([700, 500], 9000)]


@pytest.mark.parametrize("counts,N", SCALED)
@pytest.mark.parametrize("out_dtype", [lib.F32, lib.BF16])
@pytest.mark.parametrize("silu", [False, True])
def test_scales_whose_product_leaves_the_range(counts, N, out_dtype, silu):
    """Every row meets, in one of its blocks, a scale whose product with the
    weights' is subnormal, zero or infinite, next to blocks of ordinary scales
    that are all zero codes or must not notice.  Tolerance: product64's, which
    counts two scalings a block, plus 2^-125 for the one block whose scales'
    product is below the normal range, plus 2^-149 for each block's sum that ends
    there and each result that does."""
    halves, K = 2 if silu else 1, 520
    R, E, KB, NB = sum(counts), len(counts), up(520) // 128, up(N) // 128
    x, xs, w, ws, start = make(counts, N, K, halves, 31 + N)
    # block 0: huge times huge on codes of zero in every third row, else both ordinary
    # block 1: huge times huge, codes of +-2^-9 only: a normal result
    # block 2: tiny times tiny times codes near 448: a result at the end of the normal range
    # block 3: tiny times huge, the product in order
    # block 4 (8 columns): ordinary, and so the only one that counts beside block 2
    g = torch.Generator(device="cuda").manual_seed(3)
    small = torch.randint(0, 2, x.shape, generator=g, device="cuda", dtype=torch.uint8) * 128 + 1
    x[:, 0:128] = 0
    xs[0], ws[..., 0] = 2.0 ** 100, 2.0 ** 90
    x[:, 128:256] = torch.where(torch.arange(128, device="cuda") == 5, small[:, :128], 0)
    w[..., 128:256] = 1
    xs[1], ws[..., 1] = 2.0 ** 78, 2.0 ** 54     # product 2^132, block sum 2^-18: 2^114
    xs[2], ws[..., 2] = 2.0 ** -126, 2.0 ** -20  # a block sum of some 2^20: 2^-126
    xs[3], ws[..., 3] = 2.0 ** -120, 2.0 ** 110
    rows = torch.arange(R, device="cuda")
    plain = rows % 3 == 1                        # rows of the first kind: nothing but blocks 0 and 4
    x[plain, 128:512] = 0
    tiny = rows % 3 == 2                         # rows of block 2 alone
    x[tiny, 0:256], x[tiny, 384:] = 0, 0
    out = torch.full((R, N), -7.0, dtype=DT[out_dtype], device="cuda")
    say(f"[fp8] scales {counts} N={N} silu={silu} {DT[out_dtype]}")
    lib.moelora_fp8_gemm(R, N, K, E, out_dtype, lib.FP8_SILU_MUL if silu else 0, x, xs, start, w, ws, out)
    if silu:   # (values of 2^114 leave the sigmoid's range on either side: the ordinary rows count)
        keep = plain | tiny
        ref, err = product64(x, xs, w, ws, counts, N, K, True, out_dtype)
        out, ref, err = out[keep], ref[keep], err[keep]
    else:
        ref, err = product64(x, xs, w, ws, counts, N, K, False, out_dtype)
    # (bf16 below 2^-126 has steps of 2^-133)
    err = err + 2.0 ** -125 + (KB + 1) * 2.0 ** -149 + (2.0 ** -134 if out_dtype == lib.BF16 else 0)
    check(out, ref, err, out.shape[0])


@pytest.mark.parametrize("R,N", [(2, 16), (400, 16), (400, 9000)])
@pytest.mark.parametrize("out_dtype", [lib.F32, lib.BF16])
def test_one_product_at_extreme_scales(R, N, out_dtype):
    """One non-zero product a row, so the result is one number: to a step of
    float32 and half a step of the result's type, and 2^-125 where the scales'
    product is below 2^-126."""
    half = torch.finfo(DT[out_dtype]).eps / 2
    for sx, sw, cx, cw in ((2.0 ** 100, 2.0 ** 100, 0, 0x38), (2.0 ** 80, 2.0 ** 60, 1, 1),
                           (2.0 ** -126, 2.0 ** -25, 0x7e, 0x7e), (2.0 ** -126, 1.1e-4, 0x7e, 0x7e),
                           (1.1e-4, 2.0 ** -126, 0x7e, 0x7e), (2.0 ** 60, 2.0 ** 80, 1, 1),
                           (-2.0 ** 100, 2.0 ** 100, 0, 0x38), (0.0, 2.0 ** 120, 0x7e, 0x7e),
                           (2.0 ** 120, 0.0, 0x7e, 0x7e), (2.0 ** -149, 1e30, 0x7e, 0x7e)):
        x = torch.zeros(R, 128, dtype=torch.uint8, device="cuda")
        w = torch.zeros(N, 128, dtype=torch.uint8, device="cuda")
        x[:, 77], w[:, 77] = cx, cw
        out = torch.full((R, N), -7.0, dtype=DT[out_dtype], device="cuda")
        xs = torch.full((1, R), sx, device="cuda")
        ws = torch.full((up(N) // 128, 1), sw, device="cuda")
        lib.moelora_fp8_gemm(R, N, 128, 1, out_dtype, 0, x, xs, None, w, ws, out)
        want = float(TABLE[cx] * TABLE[cw]) * float(xs[0, 0]) * float(ws[0, 0])
        tol = (half + 2.0 ** -22) * abs(want) + (2.0 ** -125 if abs(sx * sw) < 2.0 ** -126 else 0) + (2.0 ** -134 if out_dtype == lib.BF16 else 2.0 ** -149)
        d = (out.double() - want).abs().max()
        assert math.isfinite(float(d)) and float(d) <= tol, (sx, sw, float(out[0, 0]), want)


def test_an_odd_scale_changes_no_other_row():
    """A row's result does not depend on whether a neighbour's scales need
    the longer way: bit for bit."""
    for counts, N in SCALED:
        for out_dtype in (lib.F32, lib.BF16):
            R, E = sum(counts), len(counts)
            x, xs, w, ws, start = make(counts, N, 384, 1, 8)
            first, second = (torch.zeros(R, N, dtype=DT[out_dtype], device="cuda") for _ in range(2))
            lib.moelora_fp8_gemm(R, N, 384, E, out_dtype, 0, x, xs, start, w, ws, first)
            xs[1, ::5] = 2.0 ** -126
            lib.moelora_fp8_gemm(R, N, 384, E, out_dtype, 0, x, xs, start, w, ws, second)
            same = [r for r in range(R) if r % 5]
            assert torch.equal(first[same], second[same])


@pytest.mark.parametrize("counts,N", SCALED)
def test_a_nan_scale_hides_no_odd_one(counts, N):
    """Rows whose scale is NaN next to rows of zero codes whose scales'
    product overflows: the latter stay what they are."""
    for out_dtype in (lib.F32, lib.BF16):
        R, E = sum(counts), len(counts)
        x, xs, w, ws, start = make(counts, N, 384, 1, 8)
        x[:, 128:256] = 0
        xs[1], ws[..., 1] = 2.0 ** 100, 2.0 ** 100
        first, second = (torch.zeros(R, N, dtype=DT[out_dtype], device="cuda") for _ in range(2))
        lib.moelora_fp8_gemm(R, N, 384, E, out_dtype, 0, x, xs, start, w, ws, first)
        assert bool(torch.isfinite(first).all())
        bad = torch.arange(R, device="cuda") // 64 % 2 == 0
        xs[1, bad] = float("nan")
        lib.moelora_fp8_gemm(R, N, 384, E, out_dtype, 0, x, xs, start, w, ws, second)
        assert bool(second[bad].isnan().all()) and torch.equal(first[~bad], second[~bad])


@pytest.mark.parametrize("R,N", [(2, 64), (40, 64), (400, 64), (400, 9000)])
@pytest.mark.parametrize("out_dtype", [lib.F32, lib.BF16])
def test_silu_over_the_range_of_gates(R, N, out_dtype):
    """Gates from -104 to 90, each one float32 product, with small and large
    up values.  float32 results: e^(-|g| / 2) to three steps of 2^-23, which
    meets the sigmoid's denominator squared and both factors of the numerator, a
    reciprocal to one step and five roundings: under 27 2^-24 of the value, here
    2^-19; and a step of the smallest subnormal for each of the three factors
    that may end there.  bf16 results: the argument of 2^x is one rounded
    product, |g| 2^-23 of the value, sigmoids below 2^-126 are zero, and the
    rounding."""
    half = torch.finfo(DT[out_dtype]).eps / 2
    x = torch.zeros(R, 128, dtype=torch.uint8, device="cuda")
    x[:, 0], x[:, 64] = 0x38, 0x38                      # 1.0 and 1.0
    w = torch.zeros(1, 2, N, 128, dtype=torch.uint8, device="cuda")
    # gate = s (1 + code), code from 0 to 0.875 in steps of 1/8; up = s' code
    eighths = torch.tensor([0, 0x20, 0x28, 0x2c, 0x30, 0x32, 0x34, 0x36], dtype=torch.uint8, device="cuda")
    at = torch.arange(N, device="cuda")
    w[0, 0, :, 0], w[0, 0, :, 64], w[0, 1, :, 0] = 0x38, eighths[at % 8], 0x38
    gate_code = 1 + TABLE.cuda()[eighths.long()][at % 8]
    xs = torch.ones(1, R, device="cuda")
    for scale in (-0.01, -1.0, -7.3, -17.7, -33.1, -47.0, -55.47, 0.01, 1.0, 20.0, 48.0):
        for up_scale in (1.0, -3.1e-3, 2.0 ** 100, 3.0 ** 70):
            ws = torch.tensor([scale, up_scale], device="cuda").view(1, 2, 1, 1).repeat(1, 1, up(N) // 128, 1)
            out = torch.full((R, N), -7.0, dtype=DT[out_dtype], device="cuda")
            lib.moelora_fp8_gemm(R, N, 128, 1, out_dtype, lib.FP8_SILU_MUL, x, xs, None, w, ws, out)
            g = (gate_code * float(ws[0, 0, 0, 0])).float().double()
            ref = g / (1 + torch.exp(-g)) * float(ws[0, 1, 0, 0])
            if out_dtype == lib.F32:
                tol = 2.0 ** -19 * ref.abs() + 3 * 2.0 ** -149
            else:
                exact = (g.abs() * 2.0 ** -23 + 2.0 ** -21) * ref.abs() + 2.0 ** -126 * (g * float(ws[0, 1, 0, 0])).abs()
                tol = half * (ref.abs() + exact) + exact + 2.0 ** -134
            d = (out.double() - ref).abs()
            assert bool((d <= tol).all()), (scale, up_scale, float((d / ref.abs()).max()) * 2.0 ** 24)


@pytest.mark.parametrize("R", [2, 400])
@pytest.mark.parametrize("out_dtype", [lib.F32, lib.BF16])
def test_silu_of_gates_that_are_not_finite(R, out_dtype):
    """A gate of +infinity gives infinity times up, and huge finite gates what
    the limit gives; a NaN gate stays NaN."""
    N = 64
    x = torch.zeros(R, 128, dtype=torch.uint8, device="cuda")
    x[:, 3] = 0x38
    w = torch.zeros(1, 2, N, 128, dtype=torch.uint8, device="cuda")
    w[:, :, :, 3] = 0x38
    xs = torch.ones(1, R, device="cuda")
    for gate, want in ((float("inf"), float("-inf")), (1e30, -2e30), (-1e30, 0.0), (float("nan"), float("nan"))):
        ws = torch.tensor([gate, -2.0], device="cuda").view(1, 2, 1, 1).contiguous()
        out = torch.full((R, N), -7.0, dtype=DT[out_dtype], device="cuda")
        lib.moelora_fp8_gemm(R, N, 128, 1, out_dtype, lib.FP8_SILU_MUL, x, xs, None, w, ws, out)
        ref = torch.full_like(out, want)
        assert torch.allclose(out, ref, rtol=torch.finfo(DT[out_dtype]).eps, atol=0, equal_nan=True), (gate, out[0, 0])


@pytest.mark.parametrize("counts,N", SCALED)
def test_rows_of_zeros(counts, N):
    """Padding rows, as the quantiser stores them (codes of zero, scale 2^-126),
    give zeros and leave the other rows what they are, bit for bit."""
    K, R, E = 384, sum(counts), len(counts)
    g = torch.Generator(device="cuda").manual_seed(N)
    _, _, w, ws, start = make(counts, N, K, 1, 9)
    v = torch.randn(R, K, generator=g, device="cuda")
    pad = torch.arange(R, device="cuda") % 3 == 1

    def run(v, dtype):
        q, s = torch.zeros(R, K, dtype=torch.uint8, device="cuda"), torch.zeros(3, R, device="cuda")
        lib.moelora_quantize_rows(R, K, lib.F32, v, R, None, 1, q, s)
        out = torch.full((R, N), -7.0, dtype=DT[dtype], device="cuda")
        lib.moelora_fp8_gemm(R, N, K, E, dtype, 0, q, s, start, w, ws, out)
        return out, s

    for dtype in (lib.F32, lib.BF16):
        full, _ = run(v, dtype)
        padded, s = run(torch.where(pad[:, None], 0.0, v), dtype)
        assert bool((s[:, pad] == 2.0 ** -126).all())
        assert bool((padded[pad] == 0).all()) and torch.equal(padded[~pad], full[~pad])
