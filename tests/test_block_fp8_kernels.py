"""Every kernel that a block-scaled product can take, on random data of several
uneven and empty experts, with odd columns and an even, an odd and a long
contraction (more than 64 blocks).  Which kernel a case takes is asserted on
the host, so a changed rule cannot quietly leave one without a case.

Beside the bound for each element (product64's), the norm of all errors is
held to what normal data give, which shows one product too many or too few:
one of K = 8300 is 1e-2 of a typical result.
  float32  some KB + 16 float32 additions, each off by at most 2^-23 of a
           partial sum no larger than the result, at random or all one way:
           under 81 2^-24 of the norm, here 2^-18.
  bf16     the last rounding, and 1.5e-5 of the result from the block sums:
           together sqrt(1 + 0.01^2) of the rounding alone, here 1.02 (SiLU
           multiplies the latter by at most 2).  Against the float32 form rounded
           to bf16, only values within that error of a border differ, each by
           a step: mean square error x step, sqrt(0.8 1.5e-5 0.8 2^-7) = 2.7e-4 of
           the norm; here 4e-4, the value at twice the error."""
import numpy as np
import pytest
import torch

from test_block_fp8 import DT, TABLE, check, codes_of, lib, make, product64, say, spread, up

ROWS = {
    "few": [2, 0, 5, 1, 0, 0, 3, 16, 17, 1, 0],
    "little": [17, 0, 33, 64, 1, 30],
    "mid": [25, 40, 0, 64, 65, 7],
    "eighty": [130, 0, 90, 127, 1, 57, 200, 129],
    "hundreds": [130, 0, 300, 127, 1, 257, 400],
    "uneven": [700, 0, 129, 1, 500, 64, 333, 250],
}
F, B = lib.F32, lib.BF16
# kernel, result types, SiLU, rows, columns, contractions
CASES = [
    ("stream1_once", (F, B), 0, "few", 70, (384, 1000, 8300)),
    ("stream1_once", (F, B), 1, "few", 70, (384, 1000, 8300)),
    ("stream1", (F, B), 0, "little", 70, (384, 1000, 8300)),
    ("stream1", (F, B), 1, "little", 70, (384, 1000, 8300)),
    ("stream2", (F, B), 0, "little", 771, (384, 1000, 8300)),
    ("stream2", (F, B), 1, "little", 300, (384, 1000, 8300)),
    ("tile2x2", (F, B), 0, "mid", 1500, (384, 1000, 8300)),
    ("tile2x2", (F, B), 1, "mid", 771, (384, 1000, 8300)),
    ("tile2x2_once", (B,), 0, "few", 6150, (384, 500)),     # (short rows only)
    ("tile2x2_once", (B,), 1, "few", 4100, (384, 500)),
    ("tile2x2_once", (F,), 0, "few", 6150, (384, 500)),
    ("tile2x4", (F, B), 0, "eighty", 1500, (384, 1000, 8300)),
    ("tile2x4", (F, B), 1, "eighty", 771, (384, 1000, 8300)),
    ("tile2x4_once", (F, B), 0, "mid", 4100, (384, 1000, 8300)),
    ("tile2x4_once", (F, B), 1, "mid", 2050, (384, 1000, 8300)),
    ("tile2x8", (B,), 0, "hundreds", 4100, (384, 1000, 8300)),
    ("tile2x8", (B,), 1, "hundreds", 2050, (384, 1000, 8300)),
    ("tile4x8", (B,), 0, "eighty", 13000, (384, 1000)),
    ("tile4x8", (B,), 0, "hundreds", 9001, (8300,)),
    ("tile4x8", (B,), 1, "eighty", 6150, (384, 1000, 8300)),
    ("tile4x4", (F,), 0, "uneven", 4100, (384, 1000, 8300)),
    ("tile4x4", (F,), 1, "uneven", 2050, (384, 1000, 8300)),
    # float32 results of few rows an expert and long ones
    ("tile2x2_once", (F,), 0, "short", 4100, (1000, 8300)),
    ("tile2x2_once", (F,), 1, "short", 2050, (1000, 8300)),
]
ROWS["short"] = ROWS["little"]
FLAT = [(k, t, s, r, n, c) for k, ts, s, r, n, cs in CASES for t in ts for c in cs]


def kernel(rows, N, K, dtype, silu):
    line = lib.moelora_fp8_gemm_info(sum(ROWS[rows]), N, K, len(ROWS[rows]), dtype, silu)
    return dict(p.split("=") for p in line.split())["kernel"]


def test_each_case_takes_its_kernel():
    for name, dtype, silu, rows, N, K in FLAT:
        assert kernel(rows, N, K, dtype, silu) == name, (rows, N, K, dtype, silu)
    common = {"stream1_once", "stream1", "stream2", "tile2x2_once", "tile2x2", "tile2x4_once", "tile2x4"}
    for dtype, own in ((F, {"tile4x4"}), (B, {"tile2x8", "tile4x8"})):
        for silu in (0, 1):
            assert {c[0] for c in FLAT if c[1] == dtype and c[2] == silu} == common | own


def test_info_refuses():
    assert lib.moelora_fp8_gemm_info(0, 8, 8, 1, F) == "kernel=none"
    for bad, want in (((-1, 8, 8, 1, F), lib.ERR_INVALID_ARG), ((4, 0, 8, 1, F), lib.ERR_UNSUPPORTED),
                      ((4, 8, 65537, 1, F), lib.ERR_UNSUPPORTED), ((4, 8, 8, 1025, F), lib.ERR_UNSUPPORTED),
                      ((4, 8, 8, 1, 2), lib.ERR_UNSUPPORTED), ((4, 8, 8, 1, F, 2), lib.ERR_UNSUPPORTED)):
        with pytest.raises(lib.MoeLoraError) as ei:
            lib.moelora_fp8_gemm_info(*bad)
        assert ei.value.status == want
    assert lib._lib.moelora_fp8_gemm_info(4, 8, 8, 1, F, 0, None, 10) == lib.ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("name,dtype,silu,rows,N,K", FLAT)
def test_kernel(name, dtype, silu, rows, N, K):
    counts = ROWS[rows]
    R, gap = sum(counts), 3
    assert kernel(rows, N, K, dtype, silu) == name
    say(f"[fp8] {name} {rows} N={N} K={K} silu={silu} {DT[dtype]}")
    x, xs, w, ws, start = make(counts, N, K, 1 + silu, N + K, gap)
    out = torch.full((R + gap, N), -7.0, dtype=DT[dtype], device="cuda")
    lib.moelora_fp8_gemm(R + gap, N, K, len(counts), dtype, silu, x, xs, start, w, ws, out)
    ref, err = product64(x, xs, w, ws, counts, N, K, silu, dtype)
    check(out, ref, err, R)
    assert bool((out[R:] == -7).all())
    out, ref = out[:R], ref[:R]
    off = float((out.double() - ref).norm() / ref.norm())
    if dtype == F:
        assert off <= 2.0 ** -18, off
        return
    rounded = float((ref.to(torch.bfloat16).double() - ref).norm() / ref.norm())
    assert off <= 1.02 * rounded, (off, rounded)
    if not silu:
        exact = torch.zeros(R + gap, N, device="cuda")
        lib.moelora_fp8_gemm(R + gap, N, K, len(counts), F, 0, x, xs, start, w, ws, exact)
        exact = exact[:R].to(torch.bfloat16).double()
        apart = float((out.double() - exact).norm() / exact.norm())
        assert apart <= 4e-4, apart


@pytest.mark.gpu
@pytest.mark.parametrize("name,dtype,silu,rows,N,K", [c for c in FLAT if c[5] == 384])
def test_kernel_with_odd_scales(name, dtype, silu, rows, N, K):
    """A block of zero codes whose two scales multiply to infinity, and one
    whose product is subnormal (off by up to 2^-125, nothing beside the rest),
    between ordinary ones: in every kernel."""
    counts = ROWS[rows]
    R = sum(counts)
    say(f"[fp8] odd scales {name} {rows} N={N} silu={silu} {DT[dtype]}")
    x, xs, w, ws, start = make(counts, N, K, 1 + silu, N + K)
    x[::2, 128:256], xs[1], ws[..., 1] = 0, 2.0 ** 100, 2.0 ** 100
    x[1::2, 128:256], xs[1, 1::2] = 1, 2.0 ** -126       # 2^-26 ordinary, small beside the rest
    xs[2, ::3] = 2.0 ** -126                              # times some 2^-6 / K^(1/2): subnormal
    out = torch.full((R, N), -7.0, dtype=DT[dtype], device="cuda")
    lib.moelora_fp8_gemm(R, N, K, len(counts), dtype, silu, x, xs, start, w, ws, out)
    ref, err = product64(x, xs, w, ws, counts, N, K, silu, dtype)
    check(out, ref, err, R)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("rows,N", [([4], 40), ([300], 900), ([900], 9000), ([90, 0, 110], 3000)])
def test_cancelling_products(rows, N, dtype):
    """Large products that cancel beside small ones, within a group of eight
    and across groups: the documented bound of the block sums, 7 2^-13 of the sum
    of magnitudes for bf16 results, float32 additions otherwise.  Scales are
    1, so the sums' errors are not hidden by the last rounding where the
    result is small."""
    K, R = 384, sum(rows)
    g = torch.Generator(device="cuda").manual_seed(N)
    start = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device="cuda")
    xs, ws = torch.ones(3, R, device="cuda"), torch.ones(len(rows), 1, up(N) // 128, 3, device="cuda")

    def f8(v):
        return v.to(torch.float8_e4m3fn).view(torch.uint8)

    def signs(*shape):
        return torch.randint(0, 2, shape, generator=g, device="cuda").float() * 2 - 1

    def binades(lo, hi, *shape):
        return torch.exp2(torch.randint(lo, hi, shape, generator=g, device="cuda").float())

    for kind in range(4):
        say(f"[fp8] cancelling {rows} N={N} kind {kind} {DT[dtype]}")
        if kind == 0:      # any binade, any sign
            x = binades(-9, 9, R, K) * signs(R, K)
            w = binades(-9, 9, len(rows), 1, N, K) * signs(len(rows), 1, N, K)
        elif kind == 1:    # 256 and -256 times 256 in one group of eight, 2^-9 .. 2^6 around
            x, w = binades(-6, 4, R, K) * signs(R, K), binades(-3, 3, len(rows), 1, N, K)
            x[:, 0::8], x[:, 5::8], w[..., 0::8], w[..., 5::8] = 256, -256, 256, 256
        elif kind == 2:    # the same, the two in groups of their own
            x, w = binades(-6, 4, R, K) * signs(R, K), binades(-3, 3, len(rows), 1, N, K)
            x[:, 0::16], x[:, 13::16], w[..., 0::16], w[..., 13::16] = 256, -256, 256, 256
        else:              # every position's products of one size, the sizes 2^-12 .. 2^16
            e = binades(-6, 9, K)
            x, w = signs(R, K) * e, signs(len(rows), 1, N, K) * e.clamp(max=256) * 1.5
        xc, wc = f8(x), f8(w.clamp(-448, 448))
        out = torch.full((R, N), -7.0, dtype=DT[dtype], device="cuda")
        lib.moelora_fp8_gemm(R, N, K, len(rows), dtype, 0, xc, xs, start, wc, ws, out)
        ref, err = product64(xc, xs, wc, ws, rows, N, K, False, dtype)
        check(out, ref, err, R)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("counts", [[40, 0, 33], [3, 1, 0, 2], [300, 0, 257, 1]])
def test_gradient_of_grouped_rows(counts, dtype):
    """dx = dy W of each expert through the transposed copy, against the formula
    on the quantised values and against the difference of <dy, y> along v."""
    N, K, E, M = 300, 200, len(counts), sum(counts)
    rng = np.random.default_rng(M)
    w = torch.from_numpy(rng.standard_normal((E, N, K), np.float32)).cuda()
    dy = torch.from_numpy(rng.standard_normal((M, N), np.float32)).cuda()
    c, ct = (torch.zeros(E, a, up(b), dtype=torch.uint8, device="cuda") for a, b in ((N, K), (K, N)))
    s, st = (torch.zeros(E, up(a) // 128, up(b) // 128, device="cuda") for a, b in ((N, K), (K, N)))
    lib.moelora_quantize_weights(E, N, K, F, w, c, s, ct, st)
    q, qs = torch.zeros(M, up(N), dtype=torch.uint8, device="cuda"), torch.zeros(up(N) // 128, M, device="cuda")
    lib.moelora_quantize_rows(M, N, F, dy, M, None, 1, q, qs)
    start = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    dx = torch.zeros(M, K, dtype=DT[dtype], device="cuda")
    lib.moelora_fp8_gemm(M, K, N, E, dtype, 0, q, qs, start, ct, st, dx)
    ref, err = product64(q, qs, ct[:, None], st[:, None], counts, K, N, False, dtype)
    check(dx, ref, err, M)
    # along v: <dx, v> = <dy, v W^T> with W from the copy that the forward reads
    table, half = TABLE.cuda(), torch.finfo(DT[dtype]).eps / 2
    v = torch.from_numpy(rng.standard_normal((M, K))).cuda()
    dyq = (table[q.long()] * qs.double().t().repeat_interleave(128, 1))[:, :N]
    lo, diff = 0, 0.0
    for e, n in enumerate(counts):
        W = (table[c[e].long()] * s[e].double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1))[:, :K]
        diff += float((dyq[lo:lo + n] * (v[lo:lo + n] @ W.t().contiguous())).sum())
        lo += n
    tol = ((err + half * (ref.abs() + err)) * v.abs()).sum()
    assert abs(float((dx.double() * v).sum()) - diff) <= float(tol)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("M,K", [(1003, 1000), (20000, 130), (5, 65536), (257, 2879)])
def test_quantize_many_rows(M, K, dtype):
    rng = np.random.default_rng(M + K)
    x = torch.from_numpy(spread(rng, M, K)).to(DT[dtype])
    codes = torch.full((M, up(K)), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((up(K) // 128, M), -1.0, device="cuda")
    say(f"[fp8] many rows M={M} K={K} {x.dtype}")
    lib.moelora_quantize_rows(M, K, dtype, x.cuda(), M, None, 1, codes, scales)
    # the smallest power of two >= max / 448, from the parts of max = m 2^e, m in [0.5, 1)
    full = np.zeros((M, up(K)))
    full[:, :K] = x.double().numpy()
    blocks = full.reshape(M, -1, 128)
    amax = np.abs(blocks).max(-1)
    m, e = np.frexp(amax)
    want = np.ldexp(1.0, np.where(amax > 0, np.maximum(e - 9 + (m > 0.875), -126), -126))
    assert np.array_equal(scales.double().cpu().numpy(), want.T)
    wc = codes_of(blocks / want[..., None]).reshape(M, -1)
    assert np.array_equal(TABLE.numpy()[codes.cpu().numpy()], TABLE.numpy()[wc])


@pytest.mark.gpu
@pytest.mark.parametrize("rows,N,K", [("few", 70, 1000), ("few", 2050, 8300), ("little", 70, 2880), ("little", 300, 384),
                                      ("one", 1100, 4096)])
def test_few_rows_are_summed_in_float32(rows, N, K):
    """Where the weights' bytes bound the product, bf16 results come from the
    exact products too: the float32 results, rounded, bit for bit."""
    counts = [1] if rows == "one" else ROWS[rows]
    R, E = sum(counts), len(counts)
    names = [lib.moelora_fp8_gemm_info(R, N, K, E, t).split()[0] for t in (F, B)]
    assert names[0] == names[1] and names[0].startswith("kernel=stream1")
    x, xs, w, ws, start = make(counts, N, K, 1, N + K)
    outs = []
    for t in (F, B):
        out = torch.full((R, N), -7.0, dtype=DT[t], device="cuda")
        lib.moelora_fp8_gemm(R, N, K, E, t, 0, x, xs, start, w, ws, out)
        outs.append(out)
    assert torch.equal(outs[0].to(torch.bfloat16), outs[1])
