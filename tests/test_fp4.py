"""4-bit weights and the product on them against plain 64-bit implementations.

Codes and scales are fixed to the bit by their definition.  Product: a bf16
row times a weight is exact in float32 (8 + 2 significant bits), a float32 row is
the exact sum of three such parts; any order of float32 additions of n terms,
truncated or rounded, is off by at most n 2^-23 S, S the sum of the magnitudes
(whose parts add up to at most 1 + 2^-7 of it): n = K or 3 K, plus 16 for the
waves' sums.  The result adds half a step of its type.  SiLU has slope at most
1.1, so its product with up is off by at most 1.1 dg |u| + |silu(g)| du + 1.1 dg
du + 2^-19 |silu(g) u|, the last for the exponential and division of |g| < 30;
a sigmoid that underflows adds at most 1e-36 |g u|."""
import numpy as np
import pytest
import torch

lib = pytest.importorskip("lora_expert_gemm_amd")
pytestmark = pytest.mark.gpu

DT = {lib.F32: torch.float32, lib.BF16: torch.bfloat16}
GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
VALUE = np.concatenate([GRID, -GRID])
F, B = lib.F32, lib.BF16


def say(*a):
    print(*a, flush=True)


def up(n, m):
    return (n + m - 1) // m * m


def sizes(mats, N, K):
    nt, kb = up(N, 16) // 16, up(K, 128) // 128
    return (mats, nt, kb, 64, 16), (mats, nt, up(kb, 4) // 4, 64, 4)


def tiles(codes, scales):
    """codes [mats][N][K] of 0..15, scales [mats][N][groups] -> the two arrays
    of the header, entry by entry."""
    mats, N, K = codes.shape
    cs, ss = sizes(mats, N, K)
    c, s = np.zeros(cs, np.uint8), np.zeros(ss, np.uint8)
    full = np.zeros((mats, cs[1] * 16, cs[2] * 128), np.uint8)
    full[:, :N, :K] = codes
    groups = np.zeros((mats, cs[1] * 16, ss[2] * 16), np.uint8)
    groups[:, :N, :scales.shape[2]] = scales
    for g in range(4):
        for r in range(16):
            for i in range(16):
                at = full[:, r::16, 32 * g + 2 * i::128], full[:, r::16, 32 * g + 2 * i + 1::128]
                c[:, :, :, 16 * g + r, i] = at[0] | at[1] << 4
            for q in range(4):
                s[:, :, :, 16 * g + r, q] = groups[:, r::16, 4 * q + g::16]
    return c, s


def quantize_np(w):
    """float64 [mats][N][K] -> codes 0..15, scale codes [mats][N][groups]."""
    mats, N, K = w.shape
    ng = up(K, 32) // 32
    v = np.zeros((mats, N, ng * 32))
    v[..., :K] = w
    v = v.reshape(mats, N, ng, 32)
    fine = np.isfinite(v).all(-1)
    amax = np.where(fine, np.abs(np.where(np.isfinite(v), v, 0)).max(-1), 1.0)
    e = np.full(amax.shape, -125)
    some = amax > 0
    e[some] = np.maximum(-125, np.floor(np.log2(amax[some])).astype(int) - 4)
    for _ in range(4):
        e = np.where(amax > 6 * np.exp2(e.astype(float)), e + 1, e)
    a = np.abs(np.where(np.isfinite(v), v, 0)) / np.exp2(e.astype(float))[..., None]
    lo = np.clip(np.searchsorted(GRID, a, side="right") - 1, 0, 7)
    hi = np.minimum(lo + 1, 7)
    dl, dh = a - GRID[lo], GRID[hi] - a
    c = np.where((dh < dl) | ((dh == dl) & (lo % 2 == 1)), hi, lo)
    c = np.where((e == 126)[..., None] & (c == 6), 5, c)
    c = np.where(fine[..., None], c | np.where(np.signbit(v), 8, 0), 0)
    return c.reshape(mats, N, -1)[..., :K].astype(np.uint8), np.where(fine, e + 127, 255).astype(np.uint8)


def values(codes, scales):
    """float64 values; a scale of 255 is NaN."""
    K = codes.shape[-1]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return VALUE[codes] * np.repeat(s, 32, -1)[..., :K]


def spread(rng, *shape):
    """Normal draws over many binades, with zeros and exact ties among them."""
    v = rng.standard_normal(shape) * np.exp2(rng.integers(-6, 4, shape))
    t = rng.random(shape)
    v[t < 0.05] = 0
    pick = (t > 0.9)
    v[pick] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, -0.25, -5, -2.5], pick.sum())
    return v.astype(np.float32)


def cu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def blank(mats, N, K):
    cs, ss = sizes(mats, N, K)
    return (torch.full(cs, 0xAA, dtype=torch.uint8, device="cuda"),
            torch.full(ss, 0xAA, dtype=torch.uint8, device="cuda"))


SIZES = [(1, 1, 1), (1, 16, 128), (2, 17, 31), (3, 5, 33), (1, 33, 127), (2, 16, 129), (1, 40, 512), (1, 15, 513),
         (2, 48, 1001), (1, 130, 700), (5, 3, 64)]


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("mats,N,K", SIZES)
def test_quantize_and_back(mats, N, K, dtype):
    say(f"[fp4] weights {mats} x {N} x {K} {DT[dtype]}")
    w = torch.from_numpy(spread(np.random.default_rng(N + K), mats, N, K)).to(DT[dtype])
    codes, scales = blank(mats, N, K)
    lib.moelora_quantize_weights_fp4(mats, N, K, dtype, w.cuda(), codes, scales)
    c, s = quantize_np(w.double().numpy())
    tc, ts = tiles(c, s)
    assert np.array_equal(scales.cpu().numpy(), ts)
    # (either zero: a weight that rounds to zero may keep its sign or not)
    got = codes.cpu().numpy()
    for shift in (0, 4):
        assert np.array_equal(VALUE[got >> shift & 15], VALUE[tc >> shift & 15])
    for out in (F, B):
        back = torch.full((mats * N * K + 8,), -7.0, dtype=DT[out], device="cuda")
        lib.moelora_dequantize_weights_fp4(mats, N, K, out, codes, scales, back)
        assert np.array_equal(back[:-8].double().cpu().numpy(), values(c, s).reshape(-1))
        assert bool((back[-8:] == -7).all())


@pytest.mark.parametrize("mats,N,K", SIZES)
def test_pack(mats, N, K):
    rng = np.random.default_rng(N * K)
    c = rng.integers(0, 16, (mats, N, K)).astype(np.uint8)
    s = rng.integers(0, 256, (mats, N, up(K, 32) // 32)).astype(np.uint8)
    wide = np.full((mats, N, up(K, 2)), 0xF, np.uint8)     # the last half byte of an odd row is not read
    wide[..., :K] = c
    codes, scales = blank(mats, N, K)
    lib.moelora_pack_weights_fp4(mats, N, K, cu(wide[..., ::2] | wide[..., 1::2] << 4), cu(s), codes, scales)
    tc, ts = tiles(c, s)
    assert np.array_equal(codes.cpu().numpy(), tc) and np.array_equal(scales.cpu().numpy(), ts)


def test_every_code_and_scale_comes_back():
    """All 16 codes with all 256 scales (2^-127 among them, 255 is NaN)."""
    c = np.tile(np.arange(16, dtype=np.uint8), (1, 256, 2))
    s = np.arange(256, dtype=np.uint8).reshape(1, 256, 1)
    tc, ts = tiles(c, s)
    want = values(c, s)
    for out in (F, B):
        back = torch.zeros(1, 256, 32, dtype=DT[out], device="cuda")
        lib.moelora_dequantize_weights_fp4(1, 256, 32, out, cu(tc), cu(ts), back)
        got = back.double().cpu().numpy()
        big = np.abs(want) >= 2.0 ** 128
        assert np.array_equal(np.isnan(got), np.isnan(want))
        ok = ~np.isnan(want) & ~big
        assert np.array_equal(got[ok], want[ok]) and (got[big] == np.sign(want[big]) * np.inf).all()


@pytest.mark.parametrize("dtype", [F, B])
def test_quantize_special_values(dtype):
    """Infinities and NaN take their group along and no other; type limits,
    subnormals and groups of zeros have defined scales."""
    tiny, most = torch.finfo(DT[dtype]).tiny, torch.finfo(DT[dtype]).max
    w = torch.zeros(1, 20, 96, dtype=DT[dtype])
    w[0, 0, 3], w[0, 1, 40], w[0, 2, 95] = float("nan"), float("inf"), -float("inf")
    w[0, 0, 50], w[0, 1, 2] = 3.0, -5.0
    w[0, 3, :32] = most
    w[0, 4, 0], w[0, 4, 1] = most, -most / 2
    w[0, 5, 0], w[0, 5, 1] = tiny / 4, -tiny
    w[0, 6, 0] = 1.5 * 2.0 ** 127
    w[0, 7, 0] = 1.75 * 2.0 ** 127
    w[0, 8, 0], w[0, 8, 1] = 2.0 ** -125 * 6, 2.0 ** -126
    w[0, 9, 0], w[0, 9, 1] = 1.5, 1.515625
    w[0, 10, :32] = -0.0
    w[0, 11, 0] = 2.0 ** -124 * 1.5
    codes, scales = blank(1, 20, 96)
    lib.moelora_quantize_weights_fp4(1, 20, 96, dtype, w.cuda(), codes, scales)
    c, s = quantize_np(w.double().numpy())
    tc, ts = tiles(c, s)
    assert np.array_equal(scales.cpu().numpy(), ts)
    got = codes.cpu().numpy()
    for shift in (0, 4):
        assert np.array_equal(VALUE[got >> shift & 15], VALUE[tc >> shift & 15])
    back = torch.zeros(1, 20, 96, device="cuda")
    lib.moelora_dequantize_weights_fp4(1, 20, 96, F, codes, scales, back)
    bad = torch.isnan(back[0])
    assert bool(bad[0, :32].all()) and bool(bad[1, 32:64].all()) and bool(bad[2, 64:].all()) and int(bad.sum()) == 96
    assert bool(torch.isfinite(back[~torch.isnan(back)]).all())


# -------------------------------------------------------------- the product

def make(counts, N, K, halves, dtype, seed, gap=0):
    """Rows, tiled weights, float64 weights and ranges."""
    rng = np.random.default_rng(seed)
    E, R = len(counts), sum(counts) + gap
    c = rng.integers(0, 16, (E * halves, N, K)).astype(np.uint8)
    mid = 127 - int(round(np.log2(max(1, K)) / 2))
    s = rng.integers(mid - 3, mid + 1, (E * halves, N, up(K, 32) // 32)).astype(np.uint8)
    tc, ts = tiles(c, s)
    x = torch.from_numpy(rng.standard_normal((R, K)).astype(np.float32)).to(DT[dtype])
    start = cu(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    return x.cuda(), cu(tc), cu(ts), cu(values(c, s)), start


def product64(x, w, counts, silu):
    """float64 result and its bound before the last rounding."""
    K = x.shape[1]
    c = ((K if x.dtype == torch.bfloat16 else 3 * K) + 16) * 2.0 ** -23 * (1 + 2.0 ** -7)
    N, halves = w.shape[1], 2 if silu else 1
    ref = torch.zeros(x.shape[0], N, dtype=torch.float64, device="cuda")
    err = torch.zeros_like(ref)
    a, lo = x.double(), 0
    for e, n in enumerate(counts):
        if n == 0:
            continue
        parts = []
        for h in range(halves):
            b = w[e * halves + h]
            parts.append((a[lo:lo + n] @ b.t().contiguous(), c * (a[lo:lo + n].abs() @ b.abs().t().contiguous())))
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


def check(out, ref, err):
    half = torch.finfo(out.dtype).eps / 2
    assert not torch.isnan(out).any()
    over = (out.double() - ref).abs() - (half * (ref.abs() + err) + err)
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
    "onehot": [0] * 30 + [150, 0],
}
SHAPES = [(1, 1), (16, 128), (33, 100), (130, 300), (576, 1100), (771, 130), (512, 2880), (40, 8300), (100, 7),
          (65, 515)]


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("counts", list(COUNTS))
def test_product(counts, N, K, silu):
    cs = COUNTS[counts]
    if len(cs) * N * K > 2 ** 26:
        cs = cs[-20:] + [4]
    R, gap = sum(cs), 5
    for dtype in (F, B):
        say(f"[fp4] product {counts} N={N} K={K} silu={silu} {DT[dtype]}")
        x, tc, ts, w, start = make(cs, N, K, 2 if silu else 1, dtype, N * 7 + K, gap)
        x[R:] = float("nan")                               # rows of no expert: not part of any result
        out = torch.full((R + gap, N), -7.0, dtype=DT[dtype], device="cuda")
        lib.moelora_fp4_gemm(R + gap, N, K, len(cs), dtype, lib.FP4_SILU_MUL if silu else 0, x, start, tc, ts, out)
        ref, err = product64(x[:R], w, cs, silu)
        check(out[:R], ref, err)
        assert bool((out[R:] == -7).all())
        if len(cs) == 1:
            o2 = torch.full((R, N), -7.0, dtype=DT[dtype], device="cuda")
            lib.moelora_fp4_gemm(R, N, K, 1, dtype, lib.FP4_SILU_MUL if silu else 0, x[:R].contiguous(), None, tc,
                                 ts, o2)
            check(o2, ref, err)


@pytest.mark.parametrize("counts", [[5, 0, 9], [70, 0, 200], [900, 800, 0]])
@pytest.mark.parametrize("silu", [False, True])
def test_ranges_that_start_late(counts, silu):
    """Rows before the first expert's and behind the last one's belong to
    nobody, and stay as they were."""
    N, K, before, behind = 160, 260, 3, 7
    R = sum(counts)
    for dtype in (F, B):
        x, tc, ts, w, start = make(counts, N, K, 2 if silu else 1, dtype, 5, before + behind)
        x[:before], x[before + R:] = float("inf"), float("nan")
        out = torch.full((before + R + behind, N), -7.0, dtype=DT[dtype], device="cuda")
        lib.moelora_fp4_gemm(before + R + behind, N, K, len(counts), dtype, lib.FP4_SILU_MUL if silu else 0, x,
                             start + before, tc, ts, out)
        ref, err = product64(x[before:before + R], w, counts, silu)
        check(out[before:before + R], ref, err)
        assert bool((out[:before] == -7).all()) and bool((out[before + R:] == -7).all())


@pytest.mark.parametrize("R", [1, 16, 40, 130, 700])
@pytest.mark.parametrize("dtype", [F, B])
def test_each_product_is_exact(R, dtype):
    """One element of the row at a time: the result is the product itself, for
    every code, also of float32 rows with all 24 bits, and scales far apart."""
    K, N = 300, 16
    rng = np.random.default_rng(R)
    c = np.tile(np.arange(16, dtype=np.uint8)[:, None], (1, 1, K)).reshape(1, 16, K)
    s = np.full((1, 16, 10), 127, np.uint8)
    s[0, :, ::2] = 60
    s[0, :, 1::3] = 200
    tc, ts = tiles(c, s)
    w = values(c, s)[0]                                            # [16][K]
    at = rng.integers(0, K, R)
    x = torch.zeros(R, K, dtype=DT[dtype])
    v = torch.from_numpy(rng.standard_normal(R)).to(DT[dtype])
    x[torch.arange(R), torch.from_numpy(at)] = v
    out = torch.zeros(R, N, dtype=DT[dtype], device="cuda")
    lib.moelora_fp4_gemm(R, N, K, 1, dtype, 0, x.cuda(), None, cu(tc), cu(ts), out)
    want = torch.from_numpy(v.double().numpy()[:, None] * w[:, at].T).to(DT[dtype])
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("R", [5, 200])
def test_nan_stays_in_its_row(R):
    """A row that is not finite, or a weight row with a NaN scale, touches its
    own results only."""
    N, K = 96, 256
    for dtype in (F, B):
        x, tc, ts, w, start = make([R], N, K, 1, dtype, 3)
        x[2, 7], x[4, 255] = float("nan"), float("inf")
        # tile 1, group entry 16 g + r with g = 2, r = 4: weight row 20
        ts[0, 1, 0, 36, 1] = 255
        out = torch.zeros(R, N, dtype=DT[dtype], device="cuda")
        lib.moelora_fp4_gemm(R, N, K, 1, dtype, 0, x, None, tc, ts, out)
        fine = torch.isfinite(out)
        assert not bool(fine[2].any()) and not bool(fine[4].any()) and not bool(fine[:, 20].any())
        rest = [i for i in range(R) if i not in (2, 4)]
        cols = [i for i in range(N) if i != 20]
        assert bool(fine[rest][:, cols].all())


@pytest.mark.parametrize("starts", [
    [0, 10, 5, 20, 30], [-5, 3, 900, 12, 30], [30, 20, 10, 0, 0], [2 ** 31 - 1] * 5, [-2 ** 31, 0, 0, 0, 30]])
@pytest.mark.parametrize("R", [30, 600])
def test_bad_ranges_stay_in_bounds(starts, R):
    """Ranges that fall or point outside are clamped: the guard rows around the
    results keep their values."""
    for dtype in (F, B):
        x, tc, ts, _, _ = make([R // 4] * 4, 64, 256, 1, dtype, 9, R - R // 4 * 4)
        buf = torch.full((R + 64, 64), -7.0, dtype=DT[dtype], device="cuda")
        lib.moelora_fp4_gemm(R, 64, 256, 4, dtype, 0, x, torch.tensor(starts, dtype=torch.int32, device="cuda"), tc,
                             ts, buf[32:32 + R])
        torch.cuda.synchronize()
        assert bool((buf[:32] == -7).all()) and bool((buf[32 + R:] == -7).all())


@pytest.mark.parametrize("R", [3, 40, 700])
def test_repeats_and_replays(R):
    """Bitwise repeatable, captured or not, on another stream too."""
    cs = [R // 3, R - R // 3]
    x, tc, ts, w, start = make(cs, 320, 640, 2, B, 21)
    out = torch.zeros(R, 320, dtype=torch.bfloat16, device="cuda")

    def step(stream=None):
        lib.moelora_fp4_gemm(R, 320, 640, 2, B, lib.FP4_SILU_MUL, x, start, tc, ts, out, stream=stream)

    step()
    first = out.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = torch.cuda.Stream()
    for _ in range(3):
        for go in (graph.replay, step, lambda: step(other)):
            out.zero_()
            torch.cuda.synchronize()
            go()
            torch.cuda.synchronize()
            assert torch.equal(out, first)


def test_product_past_32_bit_offsets():
    """An expert whose weights start past 2^32 bytes, rows past 2^32 bytes."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    N, K, E = 4096, 65536, 40
    cs, ss = sizes(E, N, K)
    w = torch.zeros(cs, dtype=torch.uint8, device="cuda")
    s = torch.full(ss, 127, dtype=torch.uint8, device="cuda")
    w[:, :, -1, 48:, 15] = 0x20                        # the last column: 1.0
    for cs in ([1] * E, [900] * E):
        R = sum(cs)
        x = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
        x[:, -1] = torch.arange(R, device="cuda") % 7
        start = cu(np.concatenate([[0], np.cumsum(cs)]).astype(np.int32))
        out = torch.zeros(R, N, dtype=torch.bfloat16, device="cuda")
        lib.moelora_fp4_gemm(R, N, K, E, B, 0, x, start, w, s, out)
        assert torch.equal(out, x[:, -1:].expand(R, N))


def test_a_step_of_the_layer_and_its_router():
    """Route, order, gate_up with SiLU * up, down, combine, and back to the
    logits: the router's part of a training step with frozen 4-bit experts,
    against the same in 64 bits on the dequantised weights.  h and y are rounded
    to bf16 here and there (2^-8 of the value each, y's inputs with them), and
    products are off by some K 2^-23: per element of out at most 2^-6 S with S
    the weighted sum of magnitudes; the gradient of a weight, <dout, y>, at most
    2^-6 of its sum of magnitudes, and the logits' gradient is linear in those."""
    T, H, I, E, k = 57, 256, 200, 8, 2
    R = T * k
    rng = np.random.default_rng(11)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    wf = [torch.from_numpy((rng.standard_normal(sh) / np.sqrt(sh[-1])).astype(np.float32)).to(torch.bfloat16).cuda()
          for sh in ((2 * E, I, H), (E, H, I))]
    q, deq = [], []
    for w in wf:
        c, s = blank(*w.shape)
        lib.moelora_quantize_weights_fp4(*w.shape, B, w, c, s)
        d = torch.zeros_like(w)
        lib.moelora_dequantize_weights_fp4(*w.shape, B, c, s, d)
        q.append((c, s)), deq.append(d.double())
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    mask = cu((np.arange(T) % 9 != 4).astype(np.uint8))
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, wt = torch.zeros(T, k, **i32), torch.zeros(T, k, device="cuda")
    start, rows, pos = torch.zeros(E + 1, **i32), torch.zeros(R, **i32), torch.zeros(T, k, **i32)
    xs = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda")
    h, y = torch.zeros(R, I, dtype=torch.bfloat16, device="cuda"), torch.zeros(R, H, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    counts, sums, loss = torch.zeros(E + 1, **i32), torch.zeros(E, device="cuda"), torch.zeros(2, device="cuda")
    dout = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    dw, dl = torch.zeros(T, k, device="cuda"), torch.zeros(T, E, device="cuda")
    dloss = torch.tensor([0.5, 0.25], device="cuda")
    lib.moelora_route(T, E, k, F, 0, logits, mask, ids, wt)
    lib.moelora_balance_loss(T, E, k, F, logits, mask, ids, counts, sums, loss, None, 0)
    lib.moelora_dispatch(T, H, E, k, B, x, ids, start, rows, pos, xs, None, 0)
    lib.moelora_fp4_gemm(R, I, H, E, B, lib.FP4_SILU_MUL, xs, start, *q[0], h)
    lib.moelora_fp4_gemm(R, H, I, E, B, 0, h, start, *q[1], y)
    lib.moelora_combine(T, H, k, B, y, pos, wt, out)
    lib.moelora_combine_backward(T, H, k, B, dout, y, pos, wt, None, dw)
    lib.moelora_route_backward(T, E, k, F, 0, logits, mask, ids, wt, dw, counts, dloss, dl)
    # the same in 64 bits, differentiated by torch on the picks
    l64 = logits.double().clone().requires_grad_(True)
    live = mask.bool()
    picked = torch.gather(l64, 1, ids.long().clamp(min=0))
    w64 = torch.softmax(picked, 1) * live[:, None]
    want, S, mag = torch.zeros(T, H, dtype=torch.float64, device="cuda"), 0, torch.zeros(T, k, device="cuda").double()
    for j in range(k):
        e = ids[:, j].long().clamp(min=0)
        gu = [(deq[0][2 * e + i] @ x.double()[..., None])[..., 0] for i in range(2)]
        hj = gu[0] * torch.sigmoid(gu[0]) * gu[1]
        yj = (deq[1][e] @ hj[..., None])[..., 0]
        big = (deq[1][e].abs() @ hj.abs()[..., None])[..., 0]
        want = want + w64[:, j, None] * yj
        S = S + w64[:, j, None] * big
        mag[:, j] = (dout.double().abs() * big).sum(1) * live
    assert bool(((out.double() - want).abs() <= 2.0 ** -6 * S.detach() + 1e-30).all())
    p = torch.softmax(l64, 1) * live[:, None]
    n = int(live.sum())
    c = counts[:E].double()
    lse = torch.logsumexp(l64, 1) * live
    total = (want * dout.double()).sum() + 0.5 * E / (k * n * n) * (c * p.sum(0)).sum() + 0.25 * (lse ** 2).sum() / n
    total.backward()
    assert int(counts[E]) == n and int(counts[:E].sum()) == n * k
    tol = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    spread_w = (w64.detach() * mag).sum(1, keepdim=True)
    tol.scatter_add_(1, ids.long().clamp(min=0), w64.detach() * (mag + spread_w) * 2.0 ** -6)
    assert bool(((dl.double() - l64.grad).abs() <= tol + 1e-6).all())
