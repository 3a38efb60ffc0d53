"""Block-of-128 E4M3 quantisation and the block-scaled product against plain
64-bit implementations.

The quantisers' results are fixed to the bit by their definition.  Product: a
block's 128 products are exact in float32 (4 + 4 significant bits); any order
of float32 additions of n terms, truncated or rounded, is off by at most
n 2^-23 S, S the sum of the magnitudes, so with KB blocks (each scaled by two
products and added once) the float32 sum is off by at most (128 + KB + 4)
2^-23 S.  For bf16 results the FP8 matrix core forms the block sums: it aligns
the eight products of a group to the largest and drops what is under 2^-13 of
the largest's power of two, so each of the other seven is off by less than
2^-13 of the largest and the groups together by at most 7 2^-13 S.  The result
adds half a step of its type.  SiLU has slope at most
1.1, so its product with up is off by at most 1.1 dg |u| + |silu(g)| du + 1.1
dg du + 2^-19 |silu(g) u|, the last for a float32 exponential and division
(a few steps of 2^-24 each, and the exponent's error of |g| 2^-24 for the
|g| < 30 that occur).  A sigmoid that underflows adds at most 1e-36 |g u|."""
import numpy as np
import pytest
import torch

lib = pytest.importorskip("lora_expert_gemm_amd")
pytestmark = pytest.mark.gpu

DT = {lib.F32: torch.float32, lib.BF16: torch.bfloat16}
TABLE = torch.tensor([(-1.0 if c & 128 else 1.0) *
                      (float("nan") if c & 127 == 127 else
                       (c & 7) * 2.0 ** -9 if not c >> 3 & 15 else
                       (8 + (c & 7)) * 2.0 ** ((c >> 3 & 15) - 10)) for c in range(256)],
                     dtype=torch.float64)


def say(*a):
    print(*a, flush=True)


def up(n):
    return (n + 127) // 128 * 128


def codes_of(v):
    """float64 values of at most 448 -> E4M3 codes, nearest, ties to even
    (by counting on the ascending list of the 127 non-negative values)."""
    grid = TABLE[:127].numpy()
    a = np.abs(v)
    lo = np.clip(np.searchsorted(grid, a, side="right") - 1, 0, 126)
    hi = np.minimum(lo + 1, 126)
    dl, dh = a - grid[lo], grid[hi] - a
    c = np.where((dh < dl) | ((dh == dl) & (lo % 2 == 1)), hi, lo)
    return (c | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def scale_of(block):
    """block float64: the smallest 2^e >= max|finite| / 448, e >= -126."""
    a = np.abs(block[np.isfinite(block)])
    m = a.max() if a.size else 0.0
    e = -126
    if m > 0:
        e = max(-126, int(np.floor(np.log2(m))) - 10)
        while m > 448 * 2.0 ** e:
            e += 1
    return 2.0 ** e


def quantize_np(v):
    """float64 [M][K] -> codes [M][P], scales [KB][M]."""
    M, K = v.shape
    full = np.zeros((M, up(K)))
    full[:, :K] = v
    codes = np.zeros(full.shape, np.uint8)
    scales = np.zeros((up(K) // 128, M))
    for r in range(M):
        for b in range(up(K) // 128):
            blk = full[r, b * 128:b * 128 + 128]
            s = scale_of(blk)
            c = codes_of(np.where(np.isfinite(blk), blk, 0) / s)
            codes[r, b * 128:b * 128 + 128] = np.where(np.isfinite(blk), c, 0x7f)
            scales[b, r] = s
    return codes, scales


def spread(rng, *shape):
    """Normal draws over many binades, with zeros and exact ties among them."""
    v = rng.standard_normal(shape) * np.exp2(rng.integers(-12, 8, shape))
    v[rng.random(shape) < 0.05] = 0
    return v.astype(np.float32)


@pytest.mark.parametrize("dtype", [lib.F32, lib.BF16])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (3, 127), (5, 129), (17, 384), (33, 130), (2, 2880),
                                 (40, 1000)])
def test_quantize_rows(M, K, dtype):
    rng = np.random.default_rng(M * 1000 + K)
    x = torch.from_numpy(spread(rng, M, K)).to(DT[dtype])
    x[0, 0] = 448.0
    if K > 200:
        x[0, 128:256] = torch.tensor(np.exp2(rng.integers(-30, 0, 128)), dtype=x.dtype)
    codes = torch.full((M, up(K)), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((up(K) // 128, M), -1.0, device="cuda")
    say(f"[fp8] rows M={M} K={K} {x.dtype}")
    lib.moelora_quantize_rows(M, K, dtype, x.cuda(), M, None, 1, codes, scales)
    wc, wsc = quantize_np(x.double().numpy())
    assert np.array_equal(scales.double().cpu().numpy(), wsc)
    got = codes.cpu().numpy()
    assert np.array_equal(TABLE.numpy()[got], TABLE.numpy()[wc])   # (either zero)


def test_quantize_special_values():
    """Infinities and NaN get the NaN code and no say in the scale; type
    limits, subnormals and all-zero blocks have defined scales."""
    x = torch.zeros(8, 256)
    x[0, 3], x[0, 4], x[0, 5], x[0, 6] = float("nan"), float("inf"), -float("inf"), 2.0
    x[1, :] = torch.finfo(torch.float32).max
    x[2, 0], x[2, 1] = 1e-45, -1e-40
    x[3, 0] = torch.finfo(torch.float32).tiny
    x[4, 130] = -448.0
    x[5, :128] = float("nan")
    x[6, :128], x[6, 128:] = 448.00003, 1.75
    x[7, :3] = torch.tensor([2.0 ** -126, 2.0 ** -136, 1.5 * 2.0 ** -135])
    codes = torch.zeros(8, 256, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(2, 8, device="cuda")
    lib.moelora_quantize_rows(8, 256, lib.F32, x.cuda(), 8, None, 1, codes, scales)
    wc, wsc = quantize_np(x.double().numpy())
    assert np.array_equal(scales.double().cpu().numpy(), wsc)
    a, b = TABLE.numpy()[codes.cpu().numpy()], TABLE.numpy()[wc]
    assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.nan_to_num(a), np.nan_to_num(b))


@pytest.mark.parametrize("dtype,K", [(lib.BF16, 136), (lib.F32, 61)])
def test_quantize_gathered_rows(dtype, K):
    """sorted_rows as the index: rows of the tail (and any other index past
    the source) leave their codes and scales as they were."""
    T, k = 23, 3
    rng = np.random.default_rng(5)
    x = torch.from_numpy(spread(rng, T, K)).to(DT[dtype])
    idx = rng.permutation(T * k).astype(np.int32)
    idx[50:] = T * k
    idx[7], idx[9], idx[11] = -1, 2 ** 31 - 1, -2 ** 31
    codes = torch.full((T * k, up(K)), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((up(K) // 128, T * k), -1.0, device="cuda")
    lib.moelora_quantize_rows(T * k, K, dtype, x.cuda(), T, torch.from_numpy(idx).cuda(), k, codes,
                              scales)
    ok = (idx >= 0) & (idx // k < T)
    wc, wsc = quantize_np(x.double().numpy()[np.where(ok, idx // k, 0)])
    assert np.array_equal(TABLE.numpy()[codes.cpu().numpy()[ok]], TABLE.numpy()[wc[ok]])
    assert np.array_equal(scales.double().cpu().numpy()[:, ok], wsc[:, ok])
    assert (codes.cpu().numpy()[~ok] == 0xAA).all() and (scales.cpu().numpy()[:, ~ok] == -1).all()


@pytest.mark.parametrize("dtype", [lib.F32, lib.BF16])
@pytest.mark.parametrize("mats,N,K", [(1, 1, 1), (2, 128, 128), (3, 130, 200), (1, 77, 1001), (2, 300, 129)])
def test_quantize_weights(mats, N, K, dtype):
    rng = np.random.default_rng(N + K)
    w = torch.from_numpy(spread(rng, mats, N, K)).to(DT[dtype])
    NB, KB = up(N) // 128, up(K) // 128
    codes = torch.full((mats, N, up(K)), 0xAA, dtype=torch.uint8, device="cuda")
    codes_t = torch.full((mats, K, up(N)), 0xAA, dtype=torch.uint8, device="cuda")
    scales, scales_t = torch.zeros(mats, NB, KB, device="cuda"), torch.zeros(mats, KB, NB, device="cuda")
    say(f"[fp8] weights {mats} x {N} x {K} {w.dtype}")
    lib.moelora_quantize_weights(mats, N, K, dtype, w.cuda(), codes, scales, codes_t, scales_t)
    full = np.zeros((mats, up(N), up(K)))
    full[:, :N, :K] = w.double().numpy()
    want = np.zeros(full.shape, np.uint8)
    for m in range(mats):
        for i in range(NB):
            for j in range(KB):
                at = (m, slice(i * 128, i * 128 + 128), slice(j * 128, j * 128 + 128))
                s = scale_of(full[at])
                assert float(scales[m, i, j]) == s == float(scales_t[m, j, i])
                want[at] = codes_of(full[at] / s)
    T = TABLE.numpy()
    assert np.array_equal(T[codes.cpu().numpy()], T[want[:, :N]])
    assert np.array_equal(T[codes_t.cpu().numpy()], T[want[:, :, :K].transpose(0, 2, 1)])
    only = torch.zeros_like(codes)
    lib.moelora_quantize_weights(mats, N, K, dtype, w.cuda(), only, scales)
    assert torch.equal(only, codes)


@pytest.mark.parametrize("dtype", [lib.F32, lib.BF16])
def test_quantize_weights_special_values(dtype):
    """Elements that are not finite get the NaN code in both copies and no say
    in their block's scale; the other blocks do not notice."""
    N, K = 140, 260
    w = torch.from_numpy(spread(np.random.default_rng(1), 1, N, K)).to(DT[dtype])
    w[0, 3, 7], w[0, 100, 130], w[0, 139, 259] = float("nan"), float("inf"), -float("inf")
    w[0, 5, 9] = 1e30
    codes, codes_t = (torch.zeros(1, a, up(b), dtype=torch.uint8, device="cuda") for a, b in ((N, K), (K, N)))
    scales, scales_t = torch.zeros(1, 2, 3, device="cuda"), torch.zeros(1, 3, 2, device="cuda")
    lib.moelora_quantize_weights(1, N, K, dtype, w.cuda(), codes, scales, codes_t, scales_t)
    T, v = TABLE.numpy(), w[0].double().numpy()
    got = T[codes[0, :, :K].cpu().numpy()]
    assert np.array_equal(np.isnan(got), ~np.isfinite(v))
    assert np.array_equal(codes[0, :, :K].cpu().numpy(), codes_t[0, :, :N].cpu().numpy().T)
    for i in range(2):
        for j in range(3):
            blk = v[i * 128:i * 128 + 128, j * 128:j * 128 + 128]
            s = scale_of(blk)
            assert float(scales[0, i, j]) == s
            fine = np.isfinite(blk)
            want = T[codes_of(np.where(fine, blk, 0) / s)]
            assert np.array_equal(got[i * 128:i * 128 + 128, j * 128:j * 128 + 128][fine], want[fine])


# -------------------------------------------------------------- the product

def make(counts, N, K, halves, seed, gap=0):
    """Random codes (every E4M3 value but NaN), float32 scales, ranges."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    E, R, KB, NB = len(counts), sum(counts) + gap, up(K) // 128, up(N) // 128

    def codes(*shape):
        # normal values, so that sums cancel and no term dwarfs the others
        v = torch.randn(*shape, generator=g, device="cuda").clamp(-4, 4) * 64
        return v.to(torch.float8_e4m3fn).view(torch.uint8)

    x, w = codes(R, up(K)), codes(E, halves, N, up(K))
    x[:, K:], w[..., K:] = 0, 0
    xs = torch.exp2(torch.randn(KB, R, generator=g, device="cuda")) / 64
    ws = torch.exp2(torch.randn(E, halves, NB, KB, generator=g, device="cuda")) / 64 / max(1, K) ** 0.5
    start = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    return x, xs, w, ws, start


def product64(x, xs, w, ws, counts, N, K, silu, out_dtype):
    """float64 result and its error bound (before the last rounding)."""
    table = TABLE.cuda()
    KB = up(K) // 128
    a = table[x.long()] * xs.double().t().repeat_interleave(128, 1)
    c = (128 + KB + 4) * 2.0 ** -23 + (7 * 2.0 ** -13 if out_dtype == lib.BF16 else 0)
    ref = torch.zeros(x.shape[0], N, dtype=torch.float64, device="cuda")
    err = torch.zeros_like(ref)
    lo = 0
    for e, n in enumerate(counts):
        parts = []
        for h in range(w.shape[1]):
            b = table[w[e, h].long()] * ws[e, h].double().repeat_interleave(128, 0)[:N] \
                .repeat_interleave(128, 1)
            rows = a[lo:lo + n]
            parts.append((rows @ b.t().contiguous(), c * (rows.abs() @ b.abs().t().contiguous())))
        if silu:
            (gv, dg), (uv, du) = parts
            s = gv * torch.sigmoid(gv)
            ref[lo:lo + n] = s * uv
            err[lo:lo + n] = 1.1 * dg * uv.abs() + s.abs() * du + 1.1 * dg * du + \
                2.0 ** -19 * (s * uv).abs() + 1e-36 * (gv * uv).abs()
        else:
            ref[lo:lo + n], err[lo:lo + n] = parts[0]
        lo += n
    return ref, err


def check(out, ref, err, kept):
    half = torch.finfo(out.dtype).eps / 2
    d = (out[:kept].double() - ref[:kept]).abs()
    over = d - (half * (ref[:kept].abs() + err[:kept]) + err[:kept])
    assert not torch.isnan(out[:kept]).any()
    assert float(over.max()) <= 0, f"worst {float(over.max())}, {int((over > 0).sum())} over"


# rows of each expert: one token; decode-sized; experts without rows (first,
# last, runs of them); skewed; more experts than rows; many rows
COUNTS = {
    "dense1": [1], "dense16": [16], "dense17": [17], "dense100": [100], "dense300": [300],
    "decode": [2, 0, 5, 1, 0, 0, 3, 16, 17, 1, 0],
    "sparse": [0] * 70 + [1] + [0] * 60 + [2, 1] + [0] * 3,
    "skewed": [0, 90, 1, 0, 3, 33],
    "wide": [25, 40, 0, 64, 65, 7],
    "many": [130, 0, 300, 127, 1, 257],
    "hundreds": [3] * 300,
    "onehot": [0] * 30 + [150, 0],                 # mean of 4 rows, one expert with all of them
    "thousand": [9, 0, 17, 3, 30, 1, 8, 12] * 128,  # 1024 experts, the limit
}
SHAPES = [(1, 1), (16, 128), (33, 100), (130, 300), (576, 1100), (771, 130), (512, 2880),
          (40, 8300)]     # more than 64 blocks


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("counts", list(COUNTS))
def test_product(counts, N, K, silu):
    cs = COUNTS[counts]
    R, gap = sum(cs), 5
    for out_dtype in (lib.F32, lib.BF16):
        say(f"[fp8] product {counts} N={N} K={K} silu={silu} {DT[out_dtype]}")
        x, xs, w, ws, start = make(cs, N, K, 2 if silu else 1, N * 7 + K, gap)
        x[R:] = 0x7f                                   # rows of no expert: never read
        out = torch.full((R + gap, N), -7.0, dtype=DT[out_dtype], device="cuda")
        lib.moelora_fp8_gemm(R + gap, N, K, len(cs), out_dtype, lib.FP8_SILU_MUL if silu else 0, x,
                             xs, start, w, ws, out)
        ref, err = product64(x, xs, w, ws, cs, N, K, silu, out_dtype)
        check(out, ref, err, R)
        assert bool((out[R:] == -7).all())
        if len(cs) == 1:
            o2 = torch.full_like(out, -7.0)
            lib.moelora_fp8_gemm(R, N, K, 1, out_dtype, lib.FP8_SILU_MUL if silu else 0, x, xs[:, :R]
                                 .contiguous(), None, w, ws, o2)
            check(o2, ref, err, R)


@pytest.mark.parametrize("counts", [[5, 0, 9], [70, 0, 200], [900, 800, 0]])
@pytest.mark.parametrize("silu", [False, True])
def test_ranges_that_start_late(counts, silu):
    """Rows before the first expert's and behind the last one's belong to
    nobody: not read, left as they were."""
    N, K, before, behind = 160, 260, 3, 7
    R = sum(counts)
    for out_dtype in (lib.F32, lib.BF16):
        x, xs, w, ws, start = make(counts, N, K, 2 if silu else 1, 5, before + behind)
        x[:before], x[before + R:] = 0x7f, 0x7f
        out = torch.full((before + R + behind, N), -7.0, dtype=DT[out_dtype], device="cuda")
        lib.moelora_fp8_gemm(before + R + behind, N, K, len(counts), out_dtype,
                             lib.FP8_SILU_MUL if silu else 0, x, xs, start + before, w, ws, out)
        ref, err = product64(x[before:], xs[:, before:], w, ws, counts, N, K, silu, out_dtype)
        check(out[before:], ref, err, R)
        assert bool((out[:before] == -7).all()) and bool((out[before + R:] == -7).all())


def test_dense_sizes_on_both_sides_of_every_choice():
    """One expert, rows and columns around the borders where another kernel or
    tile takes over."""
    K = 384
    for out_dtype in (lib.F32, lib.BF16):
        for silu in (False, True):
            for R, N in ((16, 200), (17, 200), (32, 200), (33, 200), (97, 9000), (128, 9000),
                         (129, 20000), (260, 20000), (1030, 9000), (600, 300), (1030, 64), (40, 1)):
                x, xs, w, ws, _ = make([R], N, K, 2 if silu else 1, R + N)
                out = torch.full((R, N), -7.0, dtype=DT[out_dtype], device="cuda")
                lib.moelora_fp8_gemm(R, N, K, 1, out_dtype, lib.FP8_SILU_MUL if silu else 0, x, xs, None,
                                     w, ws, out)
                ref, err = product64(x, xs, w, ws, [R], N, K, silu, out_dtype)
                check(out, ref, err, R)


@pytest.mark.parametrize("K", [90, 640, 700, 769])
@pytest.mark.parametrize("skew", [False, True])
def test_few_rows_an_expert_on_both_sides_of_every_choice(K, skew):
    """Many experts with few rows: short rows take tiles where those fill the
    chip, long ones and small outputs the streamed kernel."""
    E = 48
    counts = [90] + [0] * (E - 1) if skew else [(e * 5) % 7 for e in range(E)]
    R = sum(counts)
    for out_dtype in (lib.F32, lib.BF16):
        for silu in (False, True):
            for N in (70, 1930):
                x, xs, w, ws, start = make(counts, N, K, 2 if silu else 1, R + N + K)
                out = torch.full((R, N), -7.0, dtype=DT[out_dtype], device="cuda")
                lib.moelora_fp8_gemm(R, N, K, E, out_dtype, lib.FP8_SILU_MUL if silu else 0, x, xs, start,
                                     w, ws, out)
                ref, err = product64(x, xs, w, ws, counts, N, K, silu, out_dtype)
                check(out, ref, err, R)


@pytest.mark.parametrize("counts", [[17, 0, 33, 64, 1, 30], [260, 0, 0, 1, 0], [16, 16, 16, 16], [0, 0, 100],
                                    [31, 33, 47, 49, 15, 0, 17, 1], [500] + [0] * 24])
def test_little_work_of_several_experts(counts):
    """Few column groups: an expert's row groups go to workgroups of their own,
    and fuller experts than the mean take several passes."""
    R, E = sum(counts), len(counts)
    for out_dtype in (lib.F32, lib.BF16):
        for silu in (False, True):
            for N, K in ((1, 500), (70, 1300), (900, 300)):
                x, xs, w, ws, start = make(counts, N, K, 2 if silu else 1, R + N + K)
                out = torch.full((R, N), -7.0, dtype=DT[out_dtype], device="cuda")
                lib.moelora_fp8_gemm(R, N, K, E, out_dtype, lib.FP8_SILU_MUL if silu else 0, x, xs, start,
                                     w, ws, out)
                ref, err = product64(x, xs, w, ws, counts, N, K, silu, out_dtype)
                check(out, ref, err, R)


def test_nothing_to_gather():
    """A shard without rows: every index points past the source."""
    codes = torch.full((6, 128), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((1, 6), -1.0, device="cuda")
    idx = torch.full((6,), 6, dtype=torch.int32, device="cuda")
    lib.moelora_quantize_rows(6, 100, lib.BF16, None, 0, idx, 2, codes, scales)
    out = torch.full((6, 32), -7.0, device="cuda")
    w, ws = torch.zeros(3, 32, 128, dtype=torch.uint8, device="cuda"), torch.ones(3, 1, 1, device="cuda")
    lib.moelora_fp8_gemm(6, 32, 100, 3, lib.F32, 0, codes, scales,
                         torch.zeros(4, dtype=torch.int32, device="cuda"), w, ws, out)
    assert bool((codes == 0xAA).all()) and bool((scales == -1).all()) and bool((out == -7).all())


def test_every_code():
    """Each of the 254 finite codes against each, one product at a time."""
    c = torch.tensor([i for i in range(256) if i & 127 != 127], dtype=torch.uint8, device="cuda")
    n = c.numel()
    x, w = torch.zeros(n, 128, dtype=torch.uint8, device="cuda"), torch.zeros(n, 128, dtype=torch.uint8, device="cuda")
    for at in (0, 17, 64, 127):
        x.zero_(), w.zero_()
        x[:, at], w[:, at] = c, c
        ones = torch.ones(1, n, device="cuda")
        out = torch.zeros(n, n, device="cuda")
        lib.moelora_fp8_gemm(n, n, 128, 1, lib.F32, 0, x, ones, None, w, torch.ones(2, 1, device="cuda"), out)
        v = TABLE.cuda()[c.long()]
        assert torch.equal(out.double(), v[:, None] * v[None])


def test_nan_and_inf_stay_in_their_row():
    """A NaN code, or a scale that is infinite, touches its own row only."""
    for R in (5, 200):
        x, xs, w, ws, start = make([R], 96, 256, 1, 3)
        x[2, 7] = 0x7f
        xs[1, 4] = float("inf")
        out = torch.zeros(R, 96, device="cuda")
        lib.moelora_fp8_gemm(R, 96, 256, 1, lib.F32, 0, x, xs, None, w, ws, out)
        fine = torch.isfinite(out).all(1)
        assert not bool(fine[2]) and not bool(fine[4])
        assert bool(fine[[i for i in range(R) if i not in (2, 4)]].all())


@pytest.mark.parametrize("starts", [
    [0, 10, 5, 20, 30], [-5, 3, 900, 12, 30], [30, 20, 10, 0, 0], [2 ** 31 - 1] * 5, [-2 ** 31, 0, 0, 0, 30]])
@pytest.mark.parametrize("R", [30, 600])
def test_bad_ranges_stay_in_bounds(starts, R):
    """Ranges that fall or point outside are clamped: nothing outside the
    buffers is read or written (their guard rows keep their values)."""
    x, xs, w, ws, _ = make([R // 4] * 4, 64, 256, 1, 9, R - R // 4 * 4)
    start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    buf = torch.full((R + 64, 64), -7.0, device="cuda")
    out = buf[32:32 + R]
    lib.moelora_fp8_gemm(R, 64, 256, 4, lib.F32, 0, x, xs, start, w, ws, out)
    torch.cuda.synchronize()
    assert bool((buf[:32] == -7).all()) and bool((buf[32 + R:] == -7).all())


@pytest.mark.parametrize("R", [3, 40, 700])
def test_repeats_and_replays(R):
    """Bitwise repeatable, captured or not."""
    cs = [R // 3, R - R // 3]
    x, xs, w, ws, start = make(cs, 320, 640, 2, 21)
    out = torch.zeros(R, 320, dtype=torch.bfloat16, device="cuda")

    def step():
        lib.moelora_fp8_gemm(R, 320, 640, 2, lib.BF16, lib.FP8_SILU_MUL, x, xs, start, w, ws, out)

    step()
    first = out.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
        out.zero_()
        step()
        assert torch.equal(out, first)


def test_gradient_of_the_rows():
    """dx = dy W through the transposed copy: against the formula, and
    <dx, v> against the difference of <dy, y> along v (the product is linear
    in its rows, so the difference is exact up to rounding)."""
    M, N, K = 70, 300, 200
    rng = np.random.default_rng(2)
    w = torch.from_numpy(rng.standard_normal((1, N, K), np.float32)).cuda()
    dy = torch.from_numpy(rng.standard_normal((M, N), np.float32)).cuda()
    c, ct = (torch.zeros(1, a, up(b), dtype=torch.uint8, device="cuda") for a, b in ((N, K), (K, N)))
    NB, KB = up(N) // 128, up(K) // 128
    s, st = torch.zeros(1, NB, KB, device="cuda"), torch.zeros(1, KB, NB, device="cuda")
    lib.moelora_quantize_weights(1, N, K, lib.F32, w, c, s, ct, st)
    q = torch.zeros(M, up(N), dtype=torch.uint8, device="cuda")
    qs = torch.zeros(NB, M, device="cuda")
    lib.moelora_quantize_rows(M, N, lib.F32, dy, M, None, 1, q, qs)
    dx = torch.zeros(M, K, device="cuda")
    lib.moelora_fp8_gemm(M, K, N, 1, lib.F32, 0, q, qs, None, ct, st, dx)
    table = TABLE.cuda()
    W = (table[c[0].long()] * s[0].double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1))[:, :K]
    dyq = (table[q.long()] * qs.double().t().repeat_interleave(128, 1))[:, :N]
    mag = dyq.abs() @ W.abs()
    tol = (128 + NB + 4) * 2.0 ** -23 * mag
    assert bool(((dx.double() - dyq @ W).abs() <= tol * 1.01).all())
    v = torch.from_numpy(rng.standard_normal((M, K))).cuda()
    diff = (dyq * (v @ W.t().contiguous())).sum()
    assert abs((dx.double() * v).sum() - diff) <= (tol * 1.01 * v.abs()).sum()


def test_product_past_32_bit_offsets():
    """An expert whose weights start past 2^32 bytes, rows past 2^31 bytes."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    N, K, E = 4096, 65536, 20
    w = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    ws = torch.ones(E, N // 128, K // 128, device="cuda")
    w[:, :, -1] = 0x38                                  # 1.0
    for cs in ([1] * E, [1800] * E):
        R = sum(cs)
        x = torch.zeros(R, K, dtype=torch.uint8, device="cuda")
        x[:, -1] = 0x40                                 # 2.0
        xs = torch.ones(K // 128, R, device="cuda")
        xs[-1] = torch.arange(R, device="cuda") % 7
        start = torch.tensor(np.concatenate([[0], np.cumsum(cs)]), dtype=torch.int32, device="cuda")
        out = torch.zeros(R, N, dtype=torch.bfloat16, device="cuda")
        lib.moelora_fp8_gemm(R, N, K, E, lib.BF16, 0, x, xs, start, w, ws, out)
        assert torch.equal(out, (2 * xs[-1])[:, None].expand(R, N).to(torch.bfloat16))


def test_whole_layer_against_the_fused_one():
    """dispatch, quantise, gate_up product with SiLU * up, quantise, down
    product, combine: against moelora_forward on the same weights, which are
    E4M3 values times powers of two and so exact in bf16.  x is made of E4M3
    values with one scale a token, so its quantisation is exact; then the two
    differ by E4M3's rounding of h (at most 2^-4 of each element, or half the
    smallest step, 2^-10 of the block's scale, itself at most max|h| / 224),
    the bf16 roundings of h, y and out on either side (2^-8 of the value each)
    and float32 sums: per element at most (2^-4 + 4 2^-8) S_h plus 2^-10 / 224
    max|h| S_w, with S_h = sum_j w_j sum |h| |W_d| and S_w = sum_j w_j sum |W_d|,
    plus 2^-7 S_h for the sums and for h's own inputs."""
    T, H, I, E, k = 48, 256, 384, 8, 2
    rng = np.random.default_rng(11)
    R = T * k
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    x = torch.randn(T, H).to(torch.float8_e4m3fn).float()
    x[:, 0::128] = 448.0 / 128
    x = x.to(torch.bfloat16).cuda()
    wf = [cu(rng.standard_normal(s, np.float32) / np.sqrt(s[-1]).astype(np.float32))
          for s in ((2 * E, I, H), (E, H, I))]
    table, deq, q = TABLE.cuda().float(), [], []
    for w in wf:
        m, N, K = w.shape
        c = torch.zeros(m, N, up(K), dtype=torch.uint8, device="cuda")
        s = torch.zeros(m, up(N) // 128, up(K) // 128, device="cuda")
        lib.moelora_quantize_weights(m, N, K, lib.F32, w, c, s)
        d = table[c.long()] * s.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)
        q.append((c, s)), deq.append(d[:, :, :K].contiguous())
    logits = torch.randn(T, E, device="cuda")
    top, ids = torch.topk(logits, k)
    ids, wt = ids.to(torch.int32).contiguous(), torch.softmax(top, 1).contiguous()
    # the fused layer
    plan = lib.Plan(T, H, I, E, k, 0, 0, lib.BF16)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    want = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    plan.forward(T, x, want, ws, topk_ids=ids, topk_w=wt,
                 w_gate_up=deq[0].to(torch.bfloat16), w_down=deq[1].to(torch.bfloat16))
    # the operators
    i32 = dict(dtype=torch.int32, device="cuda")
    start, rows, pos = torch.zeros(E + 1, **i32), torch.zeros(R, **i32), torch.zeros(T, k, **i32)
    lib.moelora_dispatch(T, H, E, k, lib.BF16, None, ids, start, rows, pos, None, None, 0)
    xc, xsc = torch.zeros(R, up(H), dtype=torch.uint8, device="cuda"), torch.zeros(up(H) // 128, R, device="cuda")
    lib.moelora_quantize_rows(R, H, lib.BF16, x, T, rows, k, xc, xsc)
    h = torch.zeros(R, I, dtype=torch.bfloat16, device="cuda")
    lib.moelora_fp8_gemm(R, I, H, E, lib.BF16, lib.FP8_SILU_MUL, xc, xsc, start, *q[0], h)
    hc, hsc = torch.zeros(R, up(I), dtype=torch.uint8, device="cuda"), torch.zeros(up(I) // 128, R, device="cuda")
    lib.moelora_quantize_rows(R, I, lib.BF16, h, R, None, 1, hc, hsc)
    y = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda")
    lib.moelora_fp8_gemm(R, H, I, E, lib.BF16, 0, hc, hsc, start, *q[1], y)
    out = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    lib.moelora_combine(T, H, k, lib.BF16, y, pos, wt, out)
    sh, sw = torch.zeros(T, H, device="cuda").double(), torch.zeros(T, H, device="cuda").double()
    hd = h.double()
    for j in range(k):
        wd = deq[1][ids[:, j].long()].double().abs()             # [T][H][I]
        hj = hd[pos[:, j].long()]
        sh += wt[:, j, None].double() * (wd @ hj.abs()[..., None])[..., 0]
        sw += wt[:, j, None].double() * wd.sum(-1) * hj.abs().amax(-1, keepdim=True)
    tol = (2.0 ** -4 + 4 * 2.0 ** -8 + 2.0 ** -7) * sh + 2.0 ** -10 / 224 * sw
    d = (out.double() - want.double()).abs()
    assert bool((d <= tol).all()), float((d / tol).max())
    fro = float(d.norm() / want.double().norm())
    say(f"[fp8] layer from operators: relative difference {fro:.4f}")
    assert fro < 2.0 ** -4
