"""moelora_dispatch / moelora_combine and their gradients against plain
64-bit implementations.

Tolerances.  The order and the copies are exact.  A sum of k float32 products
in any order is off by at most (k + 1) u S with u = 2^-24 and S the sum of the
magnitudes; rounding to the output type adds half a step, finfo(t).eps / 2 of
the value.  dw is a sum of H products: (H + 1) u S covers any order."""
import numpy as np
import pytest
import torch

lib = pytest.importorskip("lora_expert_gemm_amd")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {lib.F32: torch.float32, lib.BF16: torch.bfloat16}


def say(*a):
    print(*a, flush=True)


def order(ids, E):
    """expert_start, sorted_rows, row_pos by Python's stable sort."""
    flat = ids.reshape(-1)
    kept = sorted((int(e), p) for p, e in enumerate(flat) if 0 <= e < E)
    R = flat.size
    rows = np.full(R, R, np.int32)
    pos = np.full(R, -1, np.int32)
    for at, (_, p) in enumerate(kept):
        rows[at], pos[p] = p, at
    start = np.searchsorted([e for e, _ in kept], np.arange(E + 1)).astype(np.int32)
    return start, rows, pos.reshape(ids.shape)


def make_ids(kind, T, E, k, rng):
    if kind == "uniform":
        return rng.integers(0, E, (T, k)).astype(np.int32)
    if kind == "distinct":
        return np.argsort(rng.random((T, max(E, k))), 1)[:, :k].astype(np.int32)
    if kind == "dropped":   # a shard's view: most rows belong elsewhere, in many spellings
        ids = rng.integers(-2, 3 * E, (T, k)).astype(np.int32)
        ids[rng.random((T, k)) < 0.1] = np.iinfo(np.int32).min
        ids[rng.random((T, k)) < 0.1] = np.iinfo(np.int32).max
        return ids
    if kind == "one":
        return np.full((T, k), E - 1, np.int32)
    assert kind == "none"
    return np.full((T, k), -1, np.int32)


def dispatch(ids, E, x=None, dtype=lib.F32, H=None, stream=None, fill=-7):
    T, k = ids.shape
    R = T * k
    d = dict(device="cuda", dtype=torch.int32)
    start, rows, pos = torch.full((E + 1,), -9, **d), torch.full((R,), -9, **d), torch.full((T, k), -9, **d)
    xs = None
    if x is not None:
        H = x.shape[1]
        xs = torch.full((R, H), fill, dtype=x.dtype, device="cuda")
    n = lib.moelora_dispatch_workspace(T, E, k)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    gids = torch.from_numpy(ids).cuda()
    lib.moelora_dispatch(T, H or 1, E, k, dtype, x, gids, start, rows, pos, xs, ws, n, stream)
    return start, rows, pos, xs


# T, E, k: one launch up to 2800 rows; chunks of 256 rows and more above, which
# count all the ids up to 128 max(E, 128) rows
ORDERS = [(1, 1, 1), (1, 1024, 8), (3, 5, 2), (16, 32, 4), (64, 8, 2), (333, 128, 6), (2048, 7, 1),
          (2049, 7, 1), (513, 1000, 4), (6400, 32, 4), (5000, 1024, 8), (1000, 3, 32),
          (70001, 64, 5), (1400, 40, 2), (2801, 1024, 1), (933, 300, 3), (14800, 37, 8),
          (13000, 300, 4), (70001, 1024, 2), (4096, 128, 4), (16385, 128, 1)]


@pytest.mark.parametrize("kind", ["uniform", "distinct", "dropped", "one", "none"])
@pytest.mark.parametrize("T,E,k", ORDERS)
def test_order(T, E, k, kind):
    rng = np.random.default_rng(T * 31 + E)
    if kind == "distinct" and (k > E or T * E > 5e6):
        pytest.skip("fewer experts than picks")
    ids = make_ids(kind, T, E, k, rng)
    say(f"[order] T={T} E={E} k={k} {kind}")
    start, rows, pos, _ = dispatch(ids, E)
    ws, wr, wp = order(ids, E)
    assert np.array_equal(start.cpu().numpy(), ws)
    assert np.array_equal(rows.cpu().numpy(), wr)
    assert np.array_equal(pos.cpu().numpy(), wp)


def test_no_tokens():
    start, *_ = dispatch(np.zeros((0, 2), np.int32), 5)
    assert start.tolist() == [0] * 6


@pytest.mark.parametrize("dtype", [lib.F32, lib.BF16])
# H: rows of whole 16-byte chunks, of 4 bytes, and odd (2 bytes for bf16)
@pytest.mark.parametrize("T,H,E,k,kind", [
    (1, 1, 1, 1, "uniform"), (1, 2880, 32, 4, "distinct"), (16, 2880, 32, 4, "distinct"),
    (7, 77, 5, 3, "dropped"), (33, 130, 8, 2, "dropped"), (700, 264, 16, 4, "dropped"),
    (2100, 33, 16, 2, "uniform"), (900, 1030, 8, 3, "dropped"), (1500, 8, 300, 2, "uniform"),
    (400, 2050, 4, 32, "dropped"), (9, 3, 4, 2, "dropped"), (1200, 5, 4, 2, "uniform"),
    (50, 9, 4, 2, "dropped"), (5, 517, 4, 3, "dropped"),
    # one row a workgroup and one a wave in the gradients, 2048 rows and beyond
    (512, 2879, 16, 4, "dropped"), (1025, 1259, 16, 2, "dropped"), (2048, 70, 3, 1, "uniform"),
    # rows that end inside a 128-byte line, copied by one wave, several and a part of one
    (3000, 700, 16, 4, "dropped"), (2900, 100, 8, 2, "uniform"), (1500, 2887, 8, 2, "dropped")])
def test_copy_combine_and_gradients(T, H, E, k, kind, dtype):
    rng = np.random.default_rng(T + H)
    ids = make_ids(kind, T, E, k, rng)
    dt, R = DT[dtype], T * k
    say(f"[order] copy T={T} H={H} E={E} k={k} {kind} {dt}")

    def draw(*shape):
        return torch.from_numpy(rng.standard_normal(shape, np.float32)).to(dt).cuda()

    x = draw(T, H)
    start, rows, pos, xs = dispatch(ids, E, x, dtype)
    _, wr, wp = order(ids, E)
    kept = int(start[-1])
    assert np.array_equal(pos.cpu().numpy(), wp)
    src = torch.from_numpy(wr[:kept].astype(np.int64) // k).cuda()
    assert torch.equal(xs[:kept], x[src])
    assert bool((xs[kept:] == -7).all())             # rows behind the last: as they were

    ys, dout, w = draw(R, H), draw(T, H), torch.rand(T, k, device="cuda") - 0.3
    ys[kept:] = float("nan")                         # what nobody points to is never read
    ok = torch.from_numpy(wp >= 0).cuda()
    y64 = torch.where(ok[..., None], ys[pos.long().clamp(min=0)].double(), 0.0)
    half = torch.finfo(dt).eps / 2

    out = torch.full((T, H), float("nan"), dtype=dt, device="cuda")
    for weights, run in (
            (w.double(), lambda o: lib.moelora_combine(T, H, k, dtype, ys, pos, w, o)),
            (torch.ones_like(w).double(),
             lambda o: lib.moelora_dispatch_backward(T, H, k, dtype, ys, pos, o))):
        run(out)
        terms = weights[..., None] * y64
        ref, mag = terms.sum(1), terms.abs().sum(1)
        err = (out.double() - ref).abs()
        assert bool((err <= half * ref.abs() + 2 * (k + 1) * U * mag).all())
        again = torch.empty_like(out)
        run(again)
        assert torch.equal(again, out)

    dys = torch.full((R, H), -7, dtype=dt, device="cuda")
    dw = torch.full((T, k), float("nan"), device="cuda")
    lib.moelora_combine_backward(T, H, k, dtype, dout, ys, pos, w, dys, dw)
    ref = w.double()[..., None] * dout.double()[:, None]
    at = pos.long()[ok]
    assert bool(((dys[at].double() - ref[ok]).abs() <= (half + 2 * U) * ref[ok].abs() + 1e-40).all())
    assert bool((dys[kept:] == -7).all())
    prod = dout.double()[:, None] * y64
    assert bool(((dw.double() - prod.sum(-1)).abs() <= (H + 1) * U * prod.abs().sum(-1)).all())
    assert bool((dw[~ok] == 0).all())

    # one of the two alone gives the same
    dys2, dw2 = torch.full_like(dys, -7), torch.empty_like(dw)
    lib.moelora_combine_backward(T, H, k, dtype, dout, None, pos, w, dys2, None)
    lib.moelora_combine_backward(T, H, k, dtype, dout, ys, pos, None, None, dw2)
    assert torch.equal(dys2, dys) and torch.equal(dw2, dw)


def test_gradients_against_differences():
    """combine is linear in ys and in the weights, dispatch in x: differences
    along a direction, taken in 64 bits on the formula, equal <gradient,
    direction> up to the rounding of the float32 gradients."""
    T, H, E, k = 37, 100, 6, 3
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = make_ids("dropped", T, E, k, np.random.default_rng(4))
    x = torch.randn(T, H, generator=g, device="cuda")
    start, rows, pos, xs = dispatch(ids, E, x, lib.F32)
    kept, R = int(start[-1]), T * k
    ys = torch.randn(R, H, generator=g, device="cuda")
    w = torch.rand(T, k, generator=g, device="cuda")
    dout = torch.randn(T, H, generator=g, device="cuda")

    def combine64(y, wt):
        ok = (pos >= 0)[..., None]
        return (wt[..., None] * torch.where(ok, y[pos.long().clamp(min=0)], 0.0)).sum(1)

    dys, dw = torch.zeros(R, H, device="cuda"), torch.zeros(T, k, device="cuda")
    lib.moelora_combine_backward(T, H, k, lib.F32, dout, ys, pos, w, dys, dw)
    dx = torch.zeros(T, H, device="cuda")
    lib.moelora_dispatch_backward(T, H, k, lib.F32, dys, pos, dx)
    v, u = torch.randn(R, H, generator=g, device="cuda"), torch.randn(T, k, generator=g, device="cuda")
    n = H + k + 2  # roundings on the longest chain
    d = (dout.double() * (combine64((ys + 0).double() + v.double(), w.double()) -
                          combine64(ys.double(), w.double()))).sum()
    terms = dys.double() * v.double()
    assert abs(terms.sum() - d) <= 2 * n * U * terms.abs().sum()
    d = (dout.double() * (combine64(ys.double(), w.double() + u.double()) -
                          combine64(ys.double(), w.double()))).sum()
    terms = dw.double() * u.double()
    mag = (dout.double().abs()[:, None] * ys.double().abs()[pos.long().clamp(min=0)]).sum(-1)
    assert abs(terms.sum() - d) <= 2 * n * U * (mag * u.double().abs()).sum()
    # through both: ys = xs (the identity as the expert)
    z = torch.randn(T, H, generator=g, device="cuda").double()
    tok = torch.where(rows < R, rows // k, 0).long()
    zs = torch.where((rows < R)[:, None], z[tok], 0.0)
    terms = dx.double() * z
    want = (dout.double() * combine64(zs, w.double())).sum()
    assert abs(terms.sum() - want) <= 2 * n * U * (dys.double().abs() * zs.abs()).sum()
    assert kept > 0


def test_bad_positions_are_dropped():
    """row_pos entries outside [0, R) are read as dropped, never followed."""
    T, H, k = 9, 64, 2
    pos = torch.tensor(np.random.default_rng(0).integers(0, T * k, (T, k)), dtype=torch.int32).cuda()
    pos[0, 0], pos[1, 1], pos[2, 0] = T * k, 2 ** 31 - 1, -2 ** 31
    ok = (pos >= 0) & (pos < T * k)
    ys = torch.randn(T * k, H, device="cuda")
    w = torch.rand(T, k, device="cuda")
    out = torch.empty(T, H, device="cuda")
    lib.moelora_combine(T, H, k, lib.F32, ys, pos, w, out)
    safe = torch.where(ok, pos, 0).long()
    terms = torch.where(ok[..., None], (w[..., None].double() * ys[safe].double()), 0.0)
    assert bool(((out.double() - terms.sum(1)).abs() <= 2 * 3 * U * terms.abs().sum(1)).all())
    dw = torch.empty(T, k, device="cuda")
    lib.moelora_combine_backward(T, H, k, lib.F32, out, ys, pos, w, None, dw)
    assert bool((dw[~ok] == 0).all())


def test_nan_and_inf_pass_through():
    """A NaN or an infinity stays in its own token."""
    T, H, k, E = 40, 96, 2, 4
    ids = make_ids("distinct", T, E, k, np.random.default_rng(5))
    x = torch.randn(T, H, device="cuda")
    x[3, 5], x[7, 11] = float("nan"), float("inf")
    start, rows, pos, xs = dispatch(ids, E, x, lib.F32)
    out = torch.empty(T, H, device="cuda")
    lib.moelora_combine(T, H, k, lib.F32, xs, pos, torch.ones(T, k, device="cuda"), out)
    bad = ~torch.isfinite(out)
    assert bad.sum() == 2 and bool(bad[3, 5]) and bool(bad[7, 11])


def test_most_rows():
    """R = 2^24, the limit: against numpy's stable sort."""
    T, k, E = 1 << 19, 32, 1024
    ids = np.random.default_rng(12).integers(-1, E, (T, k)).astype(np.int32)
    start, rows, pos, _ = dispatch(ids, E)
    flat = ids.reshape(-1)
    key = np.where(flat >= 0, flat, E)
    want = np.argsort(key, kind="stable").astype(np.int32)
    kept = int((flat >= 0).sum())
    assert np.array_equal(start.cpu().numpy(), np.searchsorted(key[want], np.arange(E + 1)))
    got = rows.cpu().numpy()
    assert np.array_equal(got[:kept], want[:kept]) and (got[kept:] == T * k).all()
    back = pos.cpu().numpy().reshape(-1)
    assert np.array_equal(back[want[:kept]], np.arange(kept)) and (back[flat < 0] == -1).all()


@pytest.mark.parametrize("dtype", [lib.F32, lib.BF16])
@pytest.mark.parametrize("T,H", [(3, 65536), (2, 65535), (1 << 24, 4)])
def test_widest_and_longest(T, H, dtype):
    """The limits of the width (whole chunks and odd) and of the tokens: the
    copy, then the sum of one pick, give x back."""
    E = 3
    ids = np.random.default_rng(T % 97).integers(0, E, (T, 1)).astype(np.int32)
    x = torch.randn(T, H, device="cuda").to(DT[dtype])
    start, rows, pos, xs = dispatch(ids, E, x, dtype)
    out = torch.zeros_like(x)
    lib.moelora_dispatch_backward(T, H, 1, dtype, xs, pos, out)
    assert torch.equal(out, x)
    dys, dw = torch.zeros_like(x), torch.zeros(T, 1, device="cuda")
    lib.moelora_combine_backward(T, H, 1, dtype, x, xs, pos, torch.ones(T, 1, device="cuda"), dys, dw)
    assert torch.equal(dys, xs)
    mag = (x.double() ** 2).sum(1, keepdim=True)
    assert bool(((dw.double() - mag).abs() <= (H + 1) * U * mag).all())


def test_rows_past_32_bit_offsets():
    """R H past 2^32 elements: the last rows are found and written."""
    T, H, E, k = 140_000, 8192, 4, 4
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    ids = make_ids("distinct", T, E, k, np.random.default_rng(6))
    x = torch.arange(T, device="cuda", dtype=torch.float32).remainder(251).to(torch.bfloat16)
    x = x[:, None].expand(T, H).contiguous()
    start, rows, pos, xs = dispatch(ids, E, x, lib.BF16)
    R = T * k
    assert R * H > 2 ** 32
    assert torch.equal(xs[:, 0], x[rows.long() // k, 0]) and torch.equal(xs[:, -1], xs[:, 0])
    out = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    lib.moelora_combine(T, H, k, lib.BF16, xs, pos, torch.full((T, k), 0.25, device="cuda"), out)
    assert torch.equal(out, x)
    dw = torch.zeros(T, k, device="cuda")
    lib.moelora_combine_backward(T, H, k, lib.BF16, out, xs, pos, torch.ones_like(dw),
                                 torch.empty_like(xs), dw)
    assert torch.equal(dw[:, 0].double(), x[:, 0].double() ** 2 * H)


@pytest.mark.parametrize("T", [16, 1500])
def test_captured_and_replayed(T):
    """One capture of the way there and back, replayed on new inputs."""
    H, E, k = 136, 12, 4
    R = T * k
    rng = np.random.default_rng(8)
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    x, xs = torch.zeros(T, H, device="cuda"), torch.zeros(R, H, device="cuda")
    start = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    rows, pos = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros_like(ids)
    w, out, dw = torch.rand(T, k, device="cuda"), torch.zeros_like(x), torch.zeros(T, k, device="cuda")
    dys, dx = torch.zeros_like(xs), torch.zeros_like(x)
    n = lib.moelora_dispatch_workspace(T, E, k)
    ws = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")

    def step():
        lib.moelora_dispatch(T, H, E, k, lib.F32, x, ids, start, rows, pos, xs, ws, n)
        lib.moelora_combine(T, H, k, lib.F32, xs, pos, w, out)
        lib.moelora_combine_backward(T, H, k, lib.F32, out, xs, pos, w, dys, dw)
        lib.moelora_dispatch_backward(T, H, k, lib.F32, dys, pos, dx)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        new = make_ids("dropped" if i % 2 else "uniform", T, E, k, rng)
        ids.copy_(torch.from_numpy(new))
        x.copy_(torch.randn(T, H, device="cuda"))
        for t in (xs, dys):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (start, rows, pos, xs, out, dw, dx)]
        assert np.array_equal(got[0].cpu().numpy(), order(new, E)[0])
        for t in (xs, dys):
            t.zero_()
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (start, rows, pos, xs, out, dw, dx)):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    """Calls with workspaces of their own on two streams do not meet."""
    T, H, E, k = 3000, 64, 16, 4
    streams = [torch.cuda.Stream() for _ in range(2)]
    ids = [make_ids("dropped", T, E, k, np.random.default_rng(i)) for i in range(2)]
    xs = [torch.randn(T, H, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            got.append(dispatch(ids[i % 2], E, xs[i % 2], lib.F32))
    torch.cuda.synchronize()
    for i, (start, rows, pos, _) in enumerate(got):
        want = order(ids[i % 2], E)
        assert np.array_equal(start.cpu().numpy(), want[0])
        assert np.array_equal(rows.cpu().numpy(), want[1])
        assert np.array_equal(pos.cpu().numpy(), want[2])
