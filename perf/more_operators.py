"""Measured cases of the router, balance-loss and 4-bit-weight operators.

Five operators, each in its plain form (elementary torch operations) and as a
call of this repository's library (``own`` true):

``route``    the k largest of a token's router logits and their weights.
``balance``  per-expert counts, the sums of the probabilities, and the two
             losses of the router (balance, squared logsumexp).
``route_grad``  the gradient of the weights and of both losses in the logits.
``weights``  weights to 4-bit codes (E2M1, one power of two a group of 32) and
             back, from float weights or from a checkpoint's row-major codes.
``product``  the grouped product of rows and 4-bit weights, plain or with
             SiLU(gate) * up behind it.
"""
import math

import torch

own = False

F32, BF16, CODES = "f32", "bf16", "codes"


def listed():
    return [
        # one decode step of 16 sequences on 32 experts: latency
        dict(name="route-decode", op="route", T=16, E=32, k=4, dtype=F32, all=False, off=0, mask=False),
        # a training batch of 64 sequences of 1024 tokens on 256 experts,
        # weights of the full softmax, bf16 logits
        dict(name="route-batch", op="route", T=65536, E=256, k=8, dtype=BF16, all=True, off=0, mask=False),
        # one step of 256 tokens on 128 experts
        dict(name="balance-step", op="balance", T=256, E=128, k=8, dtype=F32, off=0, mask=False),
        # a padded training batch, three experts switched off, odd token count
        dict(name="balance-batch", op="balance", T=65521, E=128, k=8, dtype=F32, off=3, mask=True),
        # the router's gradient in the prefill-sized training step
        dict(name="route-grad-step", op="route_grad", T=6400, E=32, k=4, dtype=F32, all=False, off=0,
             mask=False),
        # and of the padded batch, full softmax, bf16 logits
        dict(name="route-grad-batch", op="route_grad", T=65521, E=256, k=8, dtype=BF16, all=True, off=3,
             mask=True),
        # a checkpoint's 4-bit weights of one expert of odd sizes, laid out
        dict(name="weights-pack", op="weights", mats=2, N=771, K=2050, source=CODES),
        # the bf16 weights of the 4096 x 11008 layer's gate_up, quantised
        dict(name="weights-quantize", op="weights", mats=16, N=11008, K=4096, source=BF16),
        # one token through a dense 4096 x 11008 projection
        dict(name="product-single", op="product", T=1, E=1, k=1, K=4096, N=11008, silu=False, dtype=BF16),
        # decode: about two rows an expert, every weight read once
        dict(name="product-decode", op="product", T=16, E=32, k=4, K=2880, N=2880, silu=True, dtype=BF16),
        # sizes off every tile, experts of some 20 rows, float32 rows
        dict(name="product-ragged", op="product", T=333, E=128, k=8, K=2050, N=771, silu=False, dtype=F32),
        # the prefill's gate_up product
        dict(name="product-prefill", op="product", T=6400, E=32, k=4, K=2880, N=2880, silu=True, dtype=BF16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "balance", "route_grad", "route_grad", "weights", "product", "product",
                     "product"])
    if op == "weights":
        while True:
            c = dict(op=op, mats=_log(rng, 1, 64), N=_log(rng, 33, 11008), K=_log(rng, 33, 8192),
                     source=rng.choice([F32, BF16, CODES]))
            if c["mats"] * c["N"] * c["K"] <= 8 * 11008 * 4096:
                return c
    if op == "product":
        while True:
            E = _log(rng, 1, 128)
            k = rng.randint(1, min(8, E))
            silu = rng.random() < 0.5
            c = dict(op=op, T=_log(rng, 1, 6400), E=E, k=k, K=_log(rng, 64, 8192),
                     N=_log(rng, 64, 8192), silu=silu, dtype=rng.choice([F32, BF16, BF16]))
            width = c["N"] * (2 if silu else 1)
            # (no dearer than the listed prefill, in the plain form too, whose
            # experts are all as wide as the fullest)
            if E * width * c["K"] <= 2 ** 28 and c["T"] * k * width * c["K"] <= 2e11 \
                    and c["T"] * k * max(width, c["K"]) <= 2 ** 26:
                return c
    while True:
        E = _log(rng, 2, 1024)
        k = rng.randint(1, min(8, E))
        c = dict(op=op, T=_log(rng, 1, 262144), E=E, k=k, dtype=rng.choice([F32, BF16]),
                 off=rng.choice([0, 0, min(3, E - k)]), mask=rng.random() < 0.5)
        if op != "balance":
            c["all"] = rng.random() < 0.5
        if c["T"] * E <= 65521 * 128:
            return c


# ------------------------------------------------------------------ inputs

def _dt(name):
    return torch.bfloat16 if name == BF16 else torch.float32


def _up(n, m):
    return (n + m - 1) // m * m


def _tile(v, block):
    """[mats][N][cols] of bytes, `block` a row and tile -> tiles of 16 rows,
    a row's groups of 32 weights (block / 4 bytes each, or one of each of four
    blocks) as the product reads them."""
    mats, N, cols = v.shape
    v = torch.nn.functional.pad(v, (0, _up(cols, block) - cols, 0, _up(N, 16) - N))
    nt, nb = v.shape[1] // 16, v.shape[2] // block
    if block == 64:  # codes: [tile][block][group][row][16 bytes]
        return v.view(mats, nt, 16, nb, 4, 16).permute(0, 1, 3, 4, 2, 5).contiguous()
    # scales: [tile][4 blocks][group][row][block]
    return v.view(mats, nt, 16, nb, 4, 4).permute(0, 1, 3, 5, 2, 4).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, s = case["op"], dict(case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def codes_of(mats, N, K):
        """A checkpoint's weights: two codes a byte, a scale a group of 32."""
        c = torch.randint(0, 256, (mats, N, (K + 1) // 2), generator=g, device="cuda", dtype=torch.uint8)
        # groups of the size that 1 / sqrt(K) normal weights have, a few binades apart
        e = 127 - 1 - int(round(math.log2(math.sqrt(K))))
        sc = torch.randint(e - 2, e + 1, (mats, N, (K + 31) // 32), generator=g, device="cuda",
                           dtype=torch.uint8)
        if K % 2:
            c[..., -1] &= 15
        return c, sc

    if op == "weights":
        mats, N, K = case["mats"], case["N"], case["K"]
        if case["source"] == CODES:
            s["codes"], s["scales"] = codes_of(mats, N, K)
        else:
            s["w"] = (randn(mats, N, K) / math.sqrt(K)).to(_dt(case["source"]))
        out = torch.bfloat16 if case["source"] == BF16 else torch.float32
        nt, kb = _up(N, 16) // 16, _up(K, 128) // 128
        s["t_codes"] = torch.zeros(mats, nt, kb, 1024, dtype=torch.uint8, device="cuda")
        s["t_scales"] = torch.zeros(mats, nt, _up(kb, 4) // 4, 256, dtype=torch.uint8, device="cuda")
        s["back"] = torch.zeros(mats, N, K, dtype=out, device="cuda")
        return s

    T, E, k = case["T"], case["E"], case["k"]
    logits = randn(T, E)
    logits += 0.5 * randn(E)
    if op == "product":
        K, N = case["K"], case["N"]
        top, ids = torch.topk(logits, k, dim=1)
        key, order = torch.sort(ids.view(-1), stable=True)
        s["start"] = torch.searchsorted(key, torch.arange(E + 1, device="cuda")).to(torch.int32)
        s["cap"] = int((s["start"][1:] - s["start"][:-1]).max())  # a capacity for the plain form's padded products
        s["x"] = randn(T, K).to(_dt(case["dtype"]))[order // k].contiguous()
        s["codes"], s["scales"] = codes_of(E * (2 if case["silu"] else 1), N, K)
        s["t_codes"], s["t_scales"] = _tile(s["codes"], 64), _tile(s["scales"], 16)
        s["y"] = torch.zeros(T * k, N, dtype=_dt(case["dtype"]), device="cuda")
        return s

    if case["off"]:  # experts that are switched off
        logits[:, torch.randperm(E, generator=g, device="cuda")[:case["off"]]] = -math.inf
    s["logits"] = logits.to(_dt(case["dtype"]))
    # sequences of 128 tokens padded at their ends
    s["valid"] = None
    if case["mask"]:
        length = torch.randint(32, 129, ((T + 127) // 128,), generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        s["valid"] = (t % 128 < length[t // 128]).to(torch.uint8)
    s["ids"], s["w"] = _plain_route(s)
    if op == "route":
        s["ids"], s["w"] = torch.zeros_like(s["ids"]), torch.zeros_like(s["w"])
    elif op == "balance":
        s["counts"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        s["sums"], s["loss"] = torch.zeros(E, device="cuda"), torch.zeros(2, device="cuda")
        # the most moelora_balance_loss_workspace asks for
        s["ws"] = torch.empty(4096 * (E + 2), dtype=torch.uint8, device="cuda")
    else:
        n = T if s["valid"] is None else int(s["valid"].sum())
        counts = torch.bincount(s["ids"].view(-1).long() + 1, minlength=E + 1)[1:]
        s["counts"] = torch.cat([counts, counts.new_tensor([n])]).to(torch.int32)
        s["dw"] = randn(T, k) / T
        s["dloss"] = torch.tensor([0.01, 0.001], device="cuda")
        s["dlogits"] = torch.zeros_like(s["logits"])
    return s


# --------------------------------------------------------------------- run

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import lora_expert_gemm_amd as lib
    op = s["op"]
    if op == "weights":
        mats, N, K = s["mats"], s["N"], s["K"]
        if s["source"] == CODES:
            lib.moelora_pack_weights_fp4(mats, N, K, s["codes"], s["scales"], s["t_codes"], s["t_scales"])
        else:
            lib.moelora_quantize_weights_fp4(mats, N, K, lib.BF16 if s["source"] == BF16 else lib.F32,
                                             s["w"], s["t_codes"], s["t_scales"])
        lib.moelora_dequantize_weights_fp4(mats, N, K, lib.BF16 if s["source"] == BF16 else lib.F32,
                                           s["t_codes"], s["t_scales"], s["back"])
        return s["back"]
    dt = lib.BF16 if s["dtype"] == BF16 else lib.F32
    T, E, k = s["T"], s["E"], s["k"]
    if op == "product":
        lib.moelora_fp4_gemm(T * k, s["N"], s["K"], E, dt, lib.FP4_SILU_MUL if s["silu"] else 0, s["x"],
                             s["start"], s["t_codes"], s["t_scales"], s["y"])
        return s["y"]
    if op == "balance":
        lib.moelora_balance_loss(T, E, k, dt, s["logits"], s["valid"], s["ids"], s["counts"], s["sums"],
                                 s["loss"], s["ws"], s["ws"].numel())
        return s["counts"], s["sums"], s["loss"]
    flags = lib.ROUTE_SOFTMAX_ALL if s["all"] else 0
    if op == "route":
        lib.moelora_route(T, E, k, dt, flags, s["logits"], s["valid"], s["ids"], s["w"])
        return s["ids"], s["w"]
    lib.moelora_route_backward(T, E, k, dt, flags, s["logits"], s["valid"], s["ids"], s["w"], s["dw"],
                               s["counts"], s["dloss"], s["dlogits"])
    return s["dlogits"]


def _available(s):
    """float32 logits with -inf where an expert may not be picked."""
    l = s["logits"].float()
    if s["valid"] is not None:
        l = torch.where(s["valid"][:, None] != 0, l, -math.inf)
    return l


def _softmax(l):
    """exp(l - max) / sum and the row's logsumexp (rows of -inf: zeros)."""
    m = l.amax(1, keepdim=True)
    e = torch.where(l == -math.inf, 0.0, torch.exp(l - m))
    z = e.sum(1, keepdim=True)
    return torch.where(z > 0, e / z, 0.0), torch.where(z > 0, m + torch.log(z), 0.0)


def _plain_route(s):
    l, k = _available(s), s["k"]
    top, ids = torch.sort(l, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    gone = top == -math.inf
    if s.get("all"):
        w = torch.gather(_softmax(l)[0], 1, ids)
    else:
        w = _softmax(top)[0]
    return torch.where(gone, -1, ids).to(torch.int32), torch.where(gone, 0.0, w)


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _values(codes, scales, K):
    """float32 [mats][N][K] of row-major codes and scales."""
    table = torch.tensor(E2M1, device="cuda")
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(2)[..., :K]
    sc = torch.ldexp(torch.ones((), device="cuda"), scales.int() - 127)
    return table[c.int()] * sc.repeat_interleave(32, 2)[..., :K]


def _run_plain(s):
    op = s["op"]
    if op == "weights":
        N, K = s["N"], s["K"]
        if s["source"] == CODES:
            return _values(s["codes"], s["scales"], K)
        v = torch.nn.functional.pad(s["w"].float(), (0, _up(K, 32) - K)).view(s["mats"], N, -1, 32)
        amax = v.abs().amax(-1, keepdim=True)
        m, ex = torch.frexp(amax)  # amax = m 2^ex, m in [0.5, 1): amax / 6 = (m / 0.75) 2^(ex - 3)
        e = torch.where(amax > 0, ex - 3 + (m > 0.75).to(ex.dtype), -125).clamp(min=-125)
        scale = torch.ldexp(torch.ones_like(amax), e)
        v = v / scale
        a = v.abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        v = torch.round(v / step) * step * scale
        return v.flatten(2)[..., :K].to(s["w"].dtype)
    if op == "product":
        return _plain_product(s)
    if op == "route":
        return _plain_route(s)
    E, k = s["E"], s["k"]
    p, lse = _softmax(_available(s))
    if op == "balance":
        live = p.sum(1) > 0
        n = live.sum().to(torch.int32)
        picked = s["ids"].long()[..., None] == torch.arange(E, device="cuda")
        counts = (picked.sum(1) * live[:, None]).sum(0).to(torch.int32)
        sums = p.double().sum(0)
        some = n.double().clamp(min=1)
        loss = torch.stack([E / (k * some * some) * (counts * sums).sum(),
                            lse.double().square().sum() / some])
        return torch.cat([counts, n[None]]), sums.float(), loss.float()
    n = s["counts"][E].double()
    c = (s["counts"][:E].double() - s["counts"][:E].double().mean()).float()
    a = (s["dloss"][0] * (E / (k * n * n))).float()
    z = (s["dloss"][1] * 2 / n).float()
    d = p * (a * (c - (p * c).sum(1, keepdim=True)) + z * lse)
    ok = s["ids"] >= 0
    wg = torch.where(ok, s["w"] * s["dw"], 0.0)
    total = wg.sum(1, keepdim=True)
    at = s["ids"].long().clamp(min=0)
    if s["all"]:
        d = d - p * total
        d = d.scatter_add(1, at, wg)
    else:
        d = d.scatter_add(1, at, torch.where(ok, wg - s["w"] * total, 0.0))
    return d.to(s["logits"].dtype)


def _plain_product(s):
    K, N, E, cap = s["K"], s["N"], s["E"], s["cap"]
    R = s["x"].shape[0]
    w = _values(s["codes"], s["scales"], K).view(E, -1, K)
    start = s["start"].long()
    at = (start[:-1, None] + torch.arange(cap, device="cuda")).clamp(max=R - 1)
    padded = torch.bmm(s["x"].float()[at], w.transpose(1, 2))  # [E][cap][M N], each expert as wide as the fullest
    r = torch.arange(R, device="cuda")
    e = torch.searchsorted(start, r, right=True) - 1
    y = padded[e, r - start[e]]
    if s["silu"]:
        gate, up = y[:, :N], y[:, N:]
        y = gate / (1 + torch.exp(-gate)) * up
    return y.to(s["y"].dtype)


# -------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "weights":
        n = case["mats"] * case["N"] * case["K"]
        given = {F32: 4, BF16: 2, CODES: 17 / 32}[case["source"]]
        # (the values that come back are float32 for a checkpoint's codes)
        return {"bytes": n * (given + (2 if case["source"] == BF16 else 4)), "flops": 2 * n}
    b = 2 if case["dtype"] == BF16 else 4
    T, E, k = case["T"], case["E"], case["k"]
    if op == "product":
        R, K = T * k, case["K"]
        width = case["N"] * (2 if case["silu"] else 1)
        hit = E * (1 - (1 - k / E) ** T)  # experts that some token picks
        return {"bytes": hit * width * K * 17 / 32 + R * (K + case["N"]) * b, "flops": 2 * R * width * K}
    n = T * E
    if op == "route":
        return {"bytes": n * b + 8 * T * k, "flops": n * (4 if case["all"] else 1)}
    if op == "balance":
        return {"bytes": n * b + 4 * T * k + 8 * E, "flops": 5 * n}
    return {"bytes": 2 * n * b + 12 * T * k, "flops": 10 * n}


# ------------------------------------------------------------------- exact

def _exact_probabilities(s):
    """float64 p [T][E] and logsumexp [T], zero in rows with no expert left."""
    l = s["logits"].double()
    off = torch.isinf(l)
    if s["valid"] is not None:
        off = off | (s["valid"] == 0)[:, None]
    l = l.masked_fill(off, -1e300)
    lse = torch.logsumexp(l, 1)
    live = ~off.all(1)
    p = torch.exp(l - lse[:, None]).masked_fill(off, 0.0)
    return p, lse.masked_fill(~live, 0.0), live


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "weights":
        mats, N, K = case["mats"], case["N"], case["K"]
        grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        # (results as they are returned: every value is one of that type)
        out = torch.zeros(mats, N, K, dtype=s["back"].dtype, device="cuda")
        for m in range(mats):
            for b in range(0, K, 32):
                cols = min(32, K - b)
                if case["source"] == CODES:
                    byte = s["codes"][m, :, b // 2:(b + cols + 1) // 2].long()
                    c = torch.zeros(N, byte.shape[1] * 2, dtype=torch.long, device="cuda")
                    c[:, ::2], c[:, 1::2] = byte % 16, byte // 16
                    v = grid[c % 8] * (1 - 2 * (c // 8))
                    v = v[:, :cols] * torch.exp2(s["scales"][m, :, b // 32].double() - 127)[:, None]
                else:
                    w = s["w"][m, :, b:b + cols].double()
                    most = w.abs().amax(1).clamp(min=1e-300)
                    e = torch.ceil(torch.log2(most / 6))
                    e = torch.where(torch.exp2(e - 1) * 6 >= most, e - 1, e)
                    e = torch.where(torch.exp2(e) * 6 < most, e + 1, e).clamp(min=-125)
                    u = w / torch.exp2(e)[:, None]
                    hi = torch.searchsorted(grid, u.abs().contiguous()).clamp(max=7)
                    lo = (hi - 1).clamp(min=0)
                    up, down = grid[hi] - u.abs(), u.abs() - grid[lo]
                    c = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
                    v = torch.copysign(grid[c], w) * torch.exp2(e)[:, None]
                out[m, :, b:b + cols] = v.to(out.dtype)
        return out
    E, k = case["E"], case["k"]
    if op == "product":
        K, N = case["K"], case["N"]
        grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        out = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        start = s["start"].tolist()
        halves = 2 if case["silu"] else 1
        for e in range(E):
            lo, hi = start[e], start[e + 1]
            if lo == hi:
                continue
            made = []
            for h in range(halves):
                byte = s["codes"][e * halves + h].long()
                c = torch.zeros(N, byte.shape[1] * 2, dtype=torch.long, device="cuda")
                c[:, ::2], c[:, 1::2] = byte % 16, byte // 16
                w = (grid[c % 8] * (1 - 2 * (c // 8)))[:, :K]
                sc = torch.exp2(s["scales"][e * halves + h].double() - 127)
                w = w * sc.repeat_interleave(32, 1)[:, :K]
                made.append(s["x"][lo:hi].double() @ w.t().contiguous())
            out[lo:hi] = made[0] * torch.sigmoid(made[0]) * made[1] if case["silu"] else made[0]
        return out
    p, lse, live = _exact_probabilities(s)
    if op == "route":
        left = p.clone() if case["all"] else s["logits"].double().masked_fill(p == 0, -math.inf)
        order = torch.sort(s["logits"].double().masked_fill(~live[:, None] | torch.isinf(s["logits"]), -math.inf),
                           dim=1, descending=True, stable=True)[1][:, :k]
        w = torch.gather(left, 1, order)
        if not case["all"]:
            w = torch.softmax(w, 1)
        return None, w.masked_fill(~live[:, None], 0.0)
    if op == "balance":
        n = max(1, int(live.sum()))
        ids = s["ids"].long() + 1
        counts = torch.bincount(ids[live].view(-1), minlength=E + 1)[1:].double()
        return None, p.sum(0), torch.stack([E * (counts * p.sum(0)).sum() / (k * n * n), (lse ** 2).sum() / n])
    n = int(s["counts"][E])
    c = s["counts"][:E].double()
    d = p * (float(s["dloss"][0]) * E / k / n / n * (c - (p @ c)[:, None])
             + float(s["dloss"][1]) * 2 / n * lse[:, None])
    w, dw = s["w"].double(), s["dw"].double()
    total = (w * dw).sum(1)
    for j in range(k):
        t = torch.nonzero(s["ids"][:, j] >= 0).view(-1)
        i = s["ids"][t, j].long()
        d[t, i] += w[t, j] * (dw[t, j] if case["all"] else dw[t, j] - total[t])
    if case["all"]:
        d -= p * total[:, None]
    return d
