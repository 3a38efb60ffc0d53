"""The stand-alone router, its losses and their gradient against plain 64-bit
implementations.

Picks and counts are whole numbers and have to be equal.  Bounds of the rest
(u = 2^-24, half a float32 step):
  probabilities  an exponential of d = top - l <= 0 is off by |d| u (the rounded
    difference) and 2^-22; the sum of E of them adds one rounding for each of
    the at most 16 registers and 6 lanes, and the d u of its terms weighted by p,
    at most ln(E) <= 7 of them; a division u.  Together (d + 7 + 16 + 6 + 1 + 8) u,
    taken as (d + 40) u of the value.  What underflows adds 2^-126.
  sums over tokens  n of those, p d <= 0.37, plus an addition for each of a lane's tokens and
    16 more.
  logsumexp  |lse| u for its sum, and 40 u for the logarithm's argument and value.
  gradient  each factor's bound times the others, plus the additions (k + 8 for the picks).
Results of bf16 logits are rounded once more, by at most half a step."""
import numpy as np
import pytest
import torch

lib = pytest.importorskip("lora_expert_gemm_amd")
pytestmark = pytest.mark.gpu

DT = {lib.F32: torch.float32, lib.BF16: torch.bfloat16}
U = 2.0 ** -24
ALL = lib.ROUTE_SOFTMAX_ALL


def say(*a):
    print(*a, flush=True)


def cu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def softmax64(l, mask=None):
    """p, lse and the tokens that count, of float64 logits."""
    l = np.where((l > -np.inf), l, -np.inf)
    if mask is not None:
        l = np.where(mask[:, None] != 0, l, -np.inf)
    top = l.max(1, keepdims=True)
    live = top[:, 0] > -np.inf
    with np.errstate(invalid="ignore"):
        d = np.where(l == top, 0.0, l - top)
    e = np.where(l == -np.inf, 0.0, np.exp(d))
    z = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(live, top[:, 0] + np.log(np.maximum(z[:, 0], 1e-300)), 0.0)
    return np.where(live[:, None], e / np.maximum(z, 1e-300), 0.0), lse, live, np.where(l == -np.inf, 0.0, -d)


def route64(l, k, all_, mask=None):
    """ids, weights and the weights' bounds."""
    T = l.shape[0]
    l = np.where((l > -np.inf), l, -np.inf)
    if mask is not None:
        l = np.where(mask[:, None] != 0, l, -np.inf)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(l, ids, 1)
    p, _, _, d = softmax64(l if all_ else top)
    w, d = (np.take_along_axis(v, ids, 1) if all_ else v for v in (p, d))
    gone = top == -np.inf
    tol = w * (d + 40) * U + 2.0 ** -126
    assert T == 0 or ids.shape[1] == k
    return np.where(gone, -1, ids).astype(np.int32), np.where(gone, 0.0, w), tol


def logits_of(T, E, dtype, seed, off=0, spread=1.0):
    """Logits with ties (exact, as few values repeat), experts switched off and
    the type's lowest value among them."""
    rng = np.random.default_rng(seed)
    l = rng.standard_normal((T, E)) * spread
    l[rng.random((T, E)) < 0.2] = 0.25
    l[rng.random((T, E)) < 0.05] = -0.0
    l[rng.random((T, E)) < 0.05] = 0.0
    if off:
        l[:, rng.permutation(E)[:off]] = -np.inf
    t = torch.from_numpy(l).to(DT[dtype])
    if T > 3 and E > 2:
        t[3, 1] = torch.finfo(DT[dtype]).min
    return t


def run_route(t, k, dtype, flags, mask=None):
    T, E = t.shape
    ids = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -9.0, device="cuda")
    lib.moelora_route(T, E, k, dtype, flags, t.cuda(), mask, ids, w)
    return ids, w


SIZES = [(1, 1, 1), (1, 2, 2), (3, 7, 3), (5, 16, 4), (70, 17, 17), (16, 32, 4), (257, 33, 8), (64, 64, 6),
         (33, 65, 32), (300, 128, 8), (19, 200, 5), (7, 256, 8), (45, 257, 32), (9, 512, 10), (21, 777, 32),
         (130, 1024, 8), (5000, 8, 2)]


@pytest.mark.parametrize("flags", [0, ALL])
@pytest.mark.parametrize("dtype", [lib.F32, lib.BF16])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_route(T, E, k, dtype, flags):
    say(f"[router] route T={T} E={E} k={k} {DT[dtype]} flags={flags}")
    for off in {0, min(3, E - 1), E}:
        t = logits_of(T, E, dtype, T + E, off)
        ids, w = run_route(t, k, dtype, flags)
        want, ww, tol = route64(t.double().numpy(), k, flags == ALL)
        assert np.array_equal(ids.cpu().numpy(), want)
        assert (np.abs(w.double().cpu().numpy() - ww) <= tol).all()


def test_ties_and_signed_zeros_go_to_the_lower_expert():
    for E in (4, 20, 60, 100, 250, 500, 1000):
        l = torch.zeros(3, E)
        l[0, ::2] = -0.0
        l[1, 1::2] = -0.0
        l[2, E // 2:] = 1.0
        ids, w = run_route(l, 3, lib.F32, 0)
        assert ids.tolist() == [[0, 1, 2], [0, 1, 2], [E // 2, E // 2 + 1, (E // 2 + 2) if E > 4 else 0]]
        if E > 4:
            assert torch.allclose(w, torch.full_like(w, 1 / 3), rtol=4 * U, atol=0)


@pytest.mark.parametrize("dtype", [lib.F32, lib.BF16])
def test_route_values_that_are_not_finite(dtype):
    """NaN and -inf are never picked; +inf takes all, in equal shares."""
    inf, nan = float("inf"), float("nan")
    t = torch.tensor([[1, nan, 2, -inf, 0], [nan] * 5, [-inf] * 5, [inf, 1, 2, inf, nan], [0, -inf, nan, -inf, 0],
                      [torch.finfo(DT[dtype]).min] * 5, [torch.finfo(DT[dtype]).max, 0, nan, -1, -inf]]).to(DT[dtype])
    ids, w = run_route(t, 4, dtype, 0)
    assert ids.tolist() == [[2, 0, 4, -1], [-1] * 4, [-1] * 4, [0, 3, 2, 1], [0, 4, -1, -1], [0, 1, 2, 3],
                            [0, 1, 3, -1]]
    e = np.exp([0, -1, -2])
    want = [[*(e / e.sum()), 0], [0] * 4, [0] * 4, [.5, .5, 0, 0], [.5, .5, 0, 0], [.25] * 4, [1, 0, 0, 0]]
    assert np.allclose(w.cpu().numpy(), want, rtol=44 * U, atol=0)


@pytest.mark.parametrize("E", [9, 128])
def test_masked_tokens_have_no_picks(E):
    T, k = 77, 4
    t = logits_of(T, E, lib.F32, 3)
    mask = cu((np.arange(T) % 5 != 2).astype(np.uint8) * 255)
    t[2::5] = float("nan")                      # whatever padding holds
    ids, w = run_route(t, k, lib.F32, ALL, mask)
    m = mask.cpu().numpy()
    want, ww, tol = route64(t.double().numpy(), k, True, m)
    assert np.array_equal(ids.cpu().numpy(), want) and bool((ids[2::5] == -1).all())
    assert (np.abs(w.double().cpu().numpy() - ww) <= tol).all()
    flag = torch.zeros(T, dtype=torch.bool, device="cuda")   # any one-byte type
    i2, w2 = run_route(t, k, lib.F32, 0, flag)
    assert bool((i2 == -1).all()) and bool((w2 == 0).all())


def run_balance(t, ids, dtype, mask=None):
    (T, E), k = t.shape, ids.shape[1]
    counts = torch.full((E + 1,), -9, dtype=torch.int32, device="cuda")
    sums, loss = torch.full((E,), -9.0, device="cuda"), torch.full((2,), -9.0, device="cuda")
    n = lib.moelora_balance_loss_workspace(T, E, k)
    ws = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    lib.moelora_balance_loss(T, E, k, dtype, t.cuda(), mask, ids, counts, sums, loss, ws, n)
    assert bool((ws[n:] == 0xA5).all())
    return counts, sums, loss


def check_balance(t, ids, mask, got):
    counts, sums, loss = (v.double().cpu().numpy() for v in got)
    (T, E), k = t.shape, ids.shape[1]
    m = None if mask is None else mask.cpu().numpy()
    p, lse, live, d = softmax64(t.double().numpy(), m)
    i = ids.cpu().numpy()[live]
    c = np.array([(i == e).sum() for e in range(E)]) if E < 100 else \
        np.bincount(np.where((i >= 0) & (i < E), i, E).reshape(-1), minlength=E + 1)[:E]
    n = int(live.sum())
    assert np.array_equal(counts, np.append(c, n))
    S = p.sum(0)
    tol = (p * (d + 40)).sum(0) * U + T * 2.0 ** -126 + S * (T / 8 + 16) * U
    assert (np.abs(sums - S) <= tol).all(), float((np.abs(sums - S) / tol).max())
    if n == 0:
        assert (loss == 0).all()
        return
    l0, l1 = E / (k * n * n) * (c * S).sum(), (lse ** 2).sum() / n
    t0 = E / (k * n * n) * (c * tol).sum() + 4 * U * l0
    t1 = (2 * np.abs(lse) * (np.abs(lse) + 40) * U).sum() / n + l1 * (T / 8 + 20) * U
    # (a token left with the type's lowest value alone has an lse of -2^128, whose square float32 has only
    # as an infinity: it is above 2^255, the type ends at 2^128)
    fits = abs(loss[1] - l1) <= t1 if l1 < 2.0 ** 127 else loss[1] == np.inf
    assert abs(loss[0] - l0) <= t0 and fits, (loss, l0, l1)


@pytest.mark.parametrize("dtype", [lib.F32, lib.BF16])
@pytest.mark.parametrize("T,E,k", SIZES + [(3000, 40, 4), (4099, 128, 8), (9000, 300, 3), (40_000, 6, 2),
                                           (3001, 1024, 2), (20_000, 37, 4)])
def test_balance(T, E, k, dtype):
    say(f"[router] balance T={T} E={E} k={k} {DT[dtype]}")
    for off, masked in ((0, False), (min(2, E - 1), True), (E, False)):
        t = logits_of(T, E, dtype, T * 3 + E, off)
        mask = cu((np.random.default_rng(T).random(T) < 0.7).astype(np.uint8)) if masked else None
        ids, _ = run_route(t, k, dtype, 0, mask)
        check_balance(t, ids, mask, run_balance(t, ids, dtype, mask))


def test_balance_of_the_callers_own_ids():
    """The same expert twice, ids outside the range, ids of padding tokens."""
    T, E, k = 500, 12, 3
    t = logits_of(T, E, lib.F32, 1)
    rng = np.random.default_rng(2)
    ids = cu(rng.choice([-1, 0, 0, 3, 3, 11, 12, 2 ** 31 - 1, -2 ** 31], (T, k)).astype(np.int32))
    mask = cu((rng.random(T) < 0.5).astype(np.uint8))
    check_balance(t, ids, mask, run_balance(t, ids, lib.F32, mask))


def test_balance_of_nothing():
    """No tokens, or padding only: zeros, and nothing read."""
    E, k = 20, 2
    counts = torch.full((E + 1,), -9, dtype=torch.int32, device="cuda")
    sums, loss = torch.full((E,), -9.0, device="cuda"), torch.full((2,), -9.0, device="cuda")
    lib.moelora_balance_loss(0, E, k, lib.F32, None, None, None, counts, sums, loss, None, 0)
    assert bool((counts == 0).all()) and bool((sums == 0).all()) and bool((loss == 0).all())
    t = logits_of(40, E, lib.F32, 1)
    ids = torch.zeros(40, k, dtype=torch.int32, device="cuda")
    for v in run_balance(t, ids, lib.F32, torch.zeros(40, dtype=torch.uint8, device="cuda")):
        assert bool((v == 0).all())


def backward64(l, k, all_, ids, w, dw, counts, dloss, mask):
    """dlogits and their bound, both float64."""
    T, E = l.shape
    p, lse, live, d = softmax64(l, mask)
    out, tol = np.zeros((T, E)), np.zeros((T, E))
    pt = (d + 40) * U                               # relative bound of p
    if counts is not None:
        n, c = counts[-1], counts[:-1].astype(np.float64)
        c = c - c.mean()
        a, z = (dloss[0] * E / (k * n * n), dloss[1] * 2 / n) if n > 0 else (0, 0)
        cp, mag = p @ c, p @ np.abs(c)
        g = a * (c - cp[:, None]) + z * lse[:, None]
        # (the counts may be taken relative to any whole number: one near their mean)
        size = np.abs(a) * (np.abs(c) + 1 + mag[:, None]) + np.abs(z * lse)[:, None]
        out += p * g
        tol += p * (np.abs(g) * pt + size * 12 * U + np.abs(a) * ((p * pt) @ (np.abs(c) + 1))[:, None]
                    + np.abs(z) * 40 * U)
    if dw is not None:
        ok = (ids >= 0) & (ids < E)
        wg = np.where(ok, w * np.where(ok, dw, 0), 0.0)
        tot, mag = wg.sum(1), np.abs(wg).sum(1)
        for j in range(k):
            r = np.nonzero(ok[:, j])[0]
            v = wg[r, j] - (0 if all_ else w[r, j] * tot[r])
            np.add.at(out, (r, ids[r, j]), v)
            np.add.at(tol, (r, ids[r, j]), (np.abs(wg[r, j]) + np.abs(w[r, j]) * mag[r]) * (k + 12) * U)
        if all_:
            out -= p * tot[:, None]
            tol += p * (np.abs(tot)[:, None] * pt + mag[:, None] * (k + 12) * U)
    gone = ~(l > -np.inf) | ~live[:, None]
    tol += np.abs(out) * 8 * U + 2.0 ** -120
    return np.where(gone, 0, out), np.where(gone, 0, tol)


def run_backward(t, k, dtype, flags, ids, w, dw, counts, dloss, mask=None):
    d = torch.full(t.shape, -9.0, dtype=t.dtype, device="cuda")
    lib.moelora_route_backward(*t.shape, k, dtype, flags, t.cuda(), mask, ids, w, dw, counts, dloss, d)
    return d


def check_backward(d, ref, tol):
    half = torch.finfo(d.dtype).eps / 2 if d.dtype == torch.bfloat16 else 0
    got = d.double().cpu().numpy()
    over = np.abs(got - ref) - (tol + half * (np.abs(ref) + tol) + (2.0 ** -134 if half else 0))
    assert (over <= 0).all(), (float(over.max()), int((over > 0).sum()))


@pytest.mark.parametrize("flags", [0, ALL])
@pytest.mark.parametrize("dtype", [lib.F32, lib.BF16])
@pytest.mark.parametrize("T,E,k", SIZES + [(20_000, 32, 4), (4200, 300, 8)])
def test_backward(T, E, k, dtype, flags):
    say(f"[router] backward T={T} E={E} k={k} {DT[dtype]} flags={flags}")
    for off, masked in ((0, False), (min(2, E - 1), True)):
        t = logits_of(T, E, dtype, T * 5 + E, off)
        rng = np.random.default_rng(T + 1)
        mask = cu((rng.random(T) < 0.7).astype(np.uint8)) if masked else None
        ids, w = run_route(t, k, dtype, flags, mask)
        counts, _, _ = run_balance(t, ids, dtype, mask)
        dw = rng.standard_normal((T, k)).astype(np.float32)
        dw[ids.cpu().numpy() < 0] = np.nan          # a dropped row's gradient is not read
        dloss = np.array([0.7, -0.3], np.float32)
        for with_w, with_loss in ((1, 1), (1, 0), (0, 1)):
            dwt, dl = (cu(dw) if with_w else None), (cu(dloss) if with_loss else None)
            got = run_backward(t, k, dtype, flags, ids if with_w else None, w if with_w else None, dwt,
                               counts if with_loss else None, dl, mask)
            ref, tol = backward64(t.double().numpy(), k, flags == ALL, ids.cpu().numpy(), w.double().cpu().numpy(),
                                  dw.astype(np.float64) if with_w else None,
                                  counts.cpu().numpy() if with_loss else None, dloss.astype(np.float64),
                                  None if mask is None else mask.cpu().numpy())
            check_backward(got, ref, tol)


@pytest.mark.parametrize("flags", [0, ALL])
def test_backward_against_differences(flags):
    """<dlogits, v> against the central difference of the float64 losses along v,
    picks and counts held."""
    T, E, k, h = 9, 11, 3, 1e-4
    rng = np.random.default_rng(4)
    l = rng.standard_normal((T, E)).astype(np.float32)
    t = torch.from_numpy(l)
    ids, w = run_route(t, k, lib.F32, flags)
    counts, _, _ = run_balance(t, ids, lib.F32)
    dw, dloss = rng.standard_normal((T, k)).astype(np.float32), np.array([1.3, 0.4], np.float32)
    d = run_backward(t, k, lib.F32, flags, ids, w, cu(dw), counts, cu(dloss)).double().cpu().numpy()
    i, c = ids.cpu().numpy(), counts.cpu().numpy()[:-1]

    def value(x):
        p, lse, _, _ = softmax64(x)
        picked = np.take_along_axis(x, i, 1)
        wt = np.take_along_axis(p, i, 1) if flags else softmax64(picked)[0]
        return (wt * dw).sum() + dloss[0] * E / (k * T * T) * (c * p.sum(0)).sum() + dloss[1] * (lse ** 2).sum() / T

    for _ in range(6):
        v = rng.standard_normal((T, E))
        diff = (value(l + h * v) - value(l - h * v)) / (2 * h)
        # (the differences' own error: h^2 times a third derivative of order 1 per element, and rounding)
        assert abs((d * v).sum() - diff) <= np.abs(v).sum() * (h * h * 30 + 64 * U)


def test_backward_of_repeated_and_bad_ids():
    """The same expert in several slots adds up; ids outside the range add nothing."""
    T, E, k = 60, 10, 4
    rng = np.random.default_rng(7)
    t = logits_of(T, E, lib.F32, 7)
    ids = rng.choice([0, 0, 0, 4, 9, -1, 10, 11, 2 ** 31 - 1, -2 ** 31], (T, k)).astype(np.int32)
    w, dw = (rng.standard_normal((T, k)).astype(np.float32) for _ in range(2))
    for flags in (0, ALL):
        got = run_backward(t, k, lib.F32, flags, cu(ids), cu(w), cu(dw), None, None)
        ref, tol = backward64(t.double().numpy(), k, flags == ALL, ids, w.astype(float), dw.astype(float), None,
                              None, None)
        check_backward(got, ref, tol)


@pytest.mark.parametrize("flags", [0, ALL])
@pytest.mark.parametrize("dtype", [lib.F32, lib.BF16])
def test_backward_of_infinite_logits(dtype, flags):
    """Two logits of +inf share a token: p = 1/2 each, 0 elsewhere, and the logarithm of the
    sum, which is infinite, adds nothing where its loss has no gradient.  Every number here is
    a float of few bits, so the sums are exact."""
    inf, nan = float("inf"), float("nan")
    t = torch.tensor([[inf, 1, 2, inf, nan], [nan] * 5]).to(DT[dtype])
    ids, w = run_route(t, 4, dtype, flags)
    assert ids.tolist() == [[0, 3, 2, 1], [-1] * 4] and w.tolist() == [[.5, .5, 0, 0], [0] * 4]
    dw = cu(np.array([[1, 3, 5, 7], [nan] * 4], np.float32))
    counts, dloss = cu(np.array([3, 0, 0, 1, 0, 1], np.int32)), cu(np.array([1, 0], np.float32))
    by_w, by_loss = np.array([-.5, 0, 0, .5, 0]), np.array([.625, 0, 0, -.625, 0])
    for a, b in ((1, 0), (0, 1), (1, 1)):
        d = run_backward(t, 4, dtype, flags, ids, w, dw if a else None, counts if b else None, dloss if b else None)
        assert d.tolist() == [list(a * by_w + b * by_loss), [0] * 5]


def test_gradient_of_a_nearly_balanced_batch():
    """Counts of 2^20 and a few: taking off their mean leaves the few exactly, where
    c_i - sum c p in float32 would be off by 2^20 u = 0.06 of one."""
    T, E, k = 64, 32, 2
    t = logits_of(T, E, lib.F32, 5)
    t[3, 1] = 0.0
    counts = np.full(E + 1, 1 << 20)
    counts[:E] += np.arange(E) % 3 - 1
    counts[E] = (1 << 20) * E // k
    dloss = np.array([1e6, 0], np.float32)
    got = run_backward(t, k, lib.F32, 0, None, None, None, cu(counts.astype(np.int32)), cu(dloss))
    ref, tol = backward64(t.double().numpy(), k, False, None, None, None, counts, dloss.astype(float), None)
    check_backward(got, ref, tol)
    assert float(np.abs(tol).max()) < 1e-4 * float(np.abs(ref).max())


def test_router_repeats_and_replays():
    """Bitwise repeatable, captured or not, on small and large batches."""
    for T, E, k in ((40, 32, 4), (5000, 100, 6)):
        t = logits_of(T, E, lib.BF16, 9, 2).cuda()
        ids, w = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
        counts = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        sums, loss = torch.zeros(E, device="cuda"), torch.zeros(2, device="cuda")
        n = lib.moelora_balance_loss_workspace(T, E, k)
        ws = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")
        dw, dloss = torch.randn(T, k, device="cuda"), torch.ones(2, device="cuda")
        d = torch.zeros_like(t)

        def step():
            lib.moelora_route(T, E, k, lib.BF16, 0, t, None, ids, w)
            lib.moelora_balance_loss(T, E, k, lib.BF16, t, None, ids, counts, sums, loss, ws, n)
            lib.moelora_route_backward(T, E, k, lib.BF16, 0, t, None, ids, w, dw, counts, dloss, d)

        outs = (ids, w, counts, sums, loss, d)
        step()
        first = [v.clone() for v in outs]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for _ in range(3):
            for go in (graph.replay, step):
                for v in outs:
                    v.zero_()
                go()
                torch.cuda.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(outs, first))


def test_router_on_two_streams():
    """Calls that overlap, each with its own workspace."""
    T, E, k = 20_000, 64, 4
    ts = [logits_of(T, E, lib.F32, s).cuda() for s in (1, 2)]
    want = [run_balance(t.cpu(), run_route(t.cpu(), k, lib.F32, 0)[0], lib.F32) for t in ts]
    n = lib.moelora_balance_loss_workspace(T, E, k)
    streams = [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()
    got = []
    for t, st in zip(ts, streams):
        with torch.cuda.stream(st):
            o = (torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda"),
                 torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(E, device="cuda"),
                 torch.zeros(2, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda"))
            got.append(o)
    torch.cuda.synchronize()
    for _ in range(3):
        for t, st, o in zip(ts, streams, got):
            lib.moelora_route(T, E, k, lib.F32, 0, t, None, o[0], o[1], stream=st)
            lib.moelora_balance_loss(T, E, k, lib.F32, t, None, o[0], o[2], o[3], o[4], o[5], n, stream=st)
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(o[2:5], w))


def test_logits_past_32_bit_offsets():
    """2^22 + 3 tokens of 1024 experts: logits past 2^32 elements."""
    T, E, k = (1 << 22) + 3, 1024, 1
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    t = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    at = torch.arange(T, device="cuda") * 7 % E
    t.view(-1)[torch.arange(T, device="cuda") * E + at] = 3.0
    ids, w = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
    lib.moelora_route(T, E, k, lib.BF16, 0, t, None, ids, w)
    assert torch.equal(ids[:, 0].long(), at) and bool((w == 1).all())
    counts = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    sums, loss = torch.zeros(E, device="cuda"), torch.zeros(2, device="cuda")
    n = lib.moelora_balance_loss_workspace(T, E, k)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    lib.moelora_balance_loss(T, E, k, lib.BF16, t, None, ids, counts, sums, loss, ws, n)
    assert torch.equal(counts[:E].long(), torch.bincount(at, minlength=E)) and int(counts[E]) == T
    d = torch.full_like(t, -9.0)
    lib.moelora_route_backward(T, E, k, lib.BF16, 0, t, None, ids, w, w, None, None, d)
    assert float(d.abs().max()) == 0      # one pick: its weight does not move
