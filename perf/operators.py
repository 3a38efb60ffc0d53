"""Measured cases of the token-order and block-scaled FP8 operators.

Four operators, each in its plain form (elementary torch operations) and as a
call of this repository's library (``own`` true):

``dispatch``  routed rows sorted by expert, and the tokens copied into that
              order; ``dispatch_grad`` the gradient of the copy.
``combine``   expert outputs added back per token with the routing weights;
              ``combine_grad`` the gradients of the outputs and the weights.
``quantize``  rows in blocks of 128 (gathered into expert order on the way),
              ``quantize_weights`` weights in blocks of 128 x 128, plain and
              transposed.
``product``   the grouped matrix product of E4M3 rows and E4M3 weights with a
              scale per block of 128, plain or with SiLU(gate) * up behind it.
"""
import math

import torch

own = False

F32, BF16 = "f32", "bf16"


def listed():
    return [
        # one decode step of 16 sequences on 32 experts: latency
        dict(name="dispatch-decode", op="dispatch", T=16, H=2880, E=32, k=4, held=32, dtype=BF16),
        # a prefill of four prompts of 1600 tokens
        dict(name="dispatch-prefill", op="dispatch", T=6400, H=2880, E=32, k=4, held=32, dtype=BF16),
        # a training step on one of four shards of 128 experts (three rows in
        # four belong elsewhere and are dropped), odd token count
        dict(name="dispatch-grad-shard", op="dispatch_grad", T=4099, H=2048, E=128, k=8, held=32,
             dtype=F32),
        # the way back of a decode step and of the prefill
        dict(name="combine-decode", op="combine", T=64, H=4096, E=8, k=2, held=8, dtype=BF16),
        dict(name="combine-prefill", op="combine", T=6400, H=2880, E=32, k=4, held=32, dtype=BF16),
        # the backward pass of the prefill-sized training step
        dict(name="combine-grad", op="combine_grad", T=6400, H=2880, E=32, k=4, held=32, dtype=BF16),
        # the prefill's tokens into expert order as E4M3
        dict(name="quantize-prefill", op="quantize", T=6400, H=2880, E=32, k=4, held=32, dtype=BF16),
        # expert weights of the 4096 x 11008 layer, with the copy that the
        # gradient's product reads
        dict(name="quantize-weights", op="quantize_weights", E=8, N=11008, K=4096, dtype=BF16),
        # one token through a dense 4096 x 11008 projection
        dict(name="product-single", op="product", T=1, E=1, k=1, K=4096, N=11008, silu=False,
             out=BF16),
        # decode: about two rows an expert, every weight read once
        dict(name="product-decode", op="product", T=16, E=32, k=4, K=2880, N=2880, silu=True,
             out=BF16),
        # sizes off every tile, experts of some 20 rows, float32 results
        dict(name="product-ragged", op="product", T=333, E=128, k=8, K=2050, N=771, silu=False,
             out=F32),
        # the prefill's gate_up product
        dict(name="product-prefill", op="product", T=6400, E=32, k=4, K=2880, N=2880, silu=True,
             out=BF16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "quantize",
                     "quantize_weights", "product", "product", "product"])
    if op == "quantize_weights":
        while True:
            c = dict(op=op, E=_log(rng, 1, 64), N=_log(rng, 33, 11008), K=_log(rng, 33, 8192),
                     dtype=rng.choice([F32, BF16]))
            if c["E"] * c["N"] * c["K"] <= 8 * 11008 * 4096:
                return c
    if op == "product":
        while True:
            E = _log(rng, 1, 128)
            k = rng.randint(1, min(8, E))
            silu = rng.random() < 0.5
            c = dict(op=op, T=_log(rng, 1, 6400), E=E, k=k, K=_log(rng, 64, 8192),
                     N=_log(rng, 64, 8192), silu=silu, out=rng.choice([F32, BF16]))
            width = c["N"] * (2 if silu else 1)
            # (no dearer than the listed prefill, in the plain form too, whose
            # experts are all as wide as the fullest)
            if E * width * c["K"] <= 2 ** 28 and c["T"] * k * width * c["K"] <= 2e11 \
                    and c["T"] * k * max(width, c["K"]) <= 2 ** 26:
                return c
    while True:
        E = _log(rng, 1, 256)
        k = rng.randint(1, min(8, E))
        c = dict(op=op, T=_log(rng, 1, 16384), H=_log(rng, 64, 8192), E=E, k=k,
                 held=E if rng.random() < 0.5 else rng.randint(max(1, E // 4), E),
                 dtype=rng.choice([F32, BF16]))
        if c["T"] * k * c["H"] * (4 if c["dtype"] == F32 else 2) <= 6400 * 4 * 2880 * 2:
            return c


# ------------------------------------------------------------------ inputs

def _dt(name):
    return torch.bfloat16 if name == BF16 else torch.float32


def _routing(T, E, k, g):
    """top-k of noisy logits with a popularity per expert: [T][k] ids, weights."""
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits += 0.5 * torch.randn(E, generator=g, device="cuda")
    top, ids = torch.topk(logits, k, dim=1)
    return ids.to(torch.int32), torch.softmax(top, dim=1)


def _order(ids, E):
    """expert_start, sorted_rows, row_pos of routed rows (ids outside [0, E) dropped)."""
    flat = ids.reshape(-1).long()
    R = flat.numel()
    kept = (flat >= 0) & (flat < E)
    key = torch.where(kept, flat, torch.full_like(flat, E))
    ordered, order = torch.sort(key, stable=True)
    start = torch.searchsorted(ordered, torch.arange(E + 1, device=flat.device))
    pos = torch.empty_like(order)
    pos[order] = torch.arange(R, device=flat.device)
    pos = torch.where(kept, pos, torch.full_like(pos, -1))
    rows = torch.where(torch.arange(R, device=flat.device) < start[E], order,
                       torch.full_like(order, R))
    return start.to(torch.int32), rows.to(torch.int32), pos.to(torch.int32).view(ids.shape)


def _pitch(K):
    return (K + 127) // 128 * 128


def _pad(v, cols):
    return torch.nn.functional.pad(v, (0, cols - v.shape[-1])) if v.shape[-1] < cols else v


def _pow2_scale(amax):
    """The smallest power of two >= amax / 448, at least 2^-126."""
    m, ex = torch.frexp(amax)  # amax = m 2^ex, m in [0.5, 1): amax / 448 = (m / 0.875) 2^(ex - 9)
    e = torch.where(amax > 0, ex - 9 + (m > 0.875).to(ex.dtype), torch.full_like(ex, -126))
    return torch.ldexp(torch.ones_like(amax), e.clamp(min=-126))


def _quantize_rows(v):
    """float32 [M][K] -> E4M3 [M][pitch], scales [K blocks][M]."""
    M, P = v.shape[0], _pitch(v.shape[1])
    blocks = _pad(v, P).view(M, P // 128, 128)
    scale = _pow2_scale(blocks.abs().amax(-1))
    codes = (blocks / scale[..., None]).to(torch.float8_e4m3fn).view(M, P)
    return codes, scale.t().contiguous()


def _weight_blocks(w, scales_of):
    """[E][N][K] -> E4M3 [E][N][pitch(K)] and scales [E][N blocks][K blocks]."""
    E, N, K = w.shape
    NB, KB = _pitch(N) // 128, _pitch(K) // 128
    full = torch.nn.functional.pad(w, (0, KB * 128 - K, 0, NB * 128 - N)).float()
    blocks = full.view(E, NB, 128, KB, 128)
    scale = scales_of(blocks.abs().amax(4).amax(2))
    codes = (blocks / scale[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return codes.view(E, NB * 128, KB * 128), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, s = case["op"], dict(case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if op == "quantize_weights":
        E, N, K = case["E"], case["N"], case["K"]
        s["w"] = (randn(E, N, K) / math.sqrt(K)).to(_dt(case["dtype"]))
        s["codes"] = torch.zeros(E, N, _pitch(K), dtype=torch.uint8, device="cuda")
        s["codes_t"] = torch.zeros(E, K, _pitch(N), dtype=torch.uint8, device="cuda")
        NB, KB = _pitch(N) // 128, _pitch(K) // 128
        s["scales"] = torch.zeros(E, NB, KB, device="cuda")
        s["scales_t"] = torch.zeros(E, KB, NB, device="cuda")
        return s

    if op == "product":
        T, E, k, K, N = (case[n] for n in ("T", "E", "k", "K", "N"))
        R, M = T * k, 2 if case["silu"] else 1
        ids, _ = _routing(T, E, k, g)
        start, rows, _ = _order(ids, E)
        x = randn(T, K).to(torch.bfloat16).float()
        s["codes"], s["scales"] = _quantize_rows(x[(rows // k).long()])
        s["codes"] = s["codes"].view(torch.uint8)
        # a checkpoint's weights: any float32 scale, amax / 448 of each block
        halves = []
        for _ in range(M):
            codes, scale = _weight_blocks(randn(E, N, K) / math.sqrt(K),
                                          lambda amax: (amax / 448).clamp(min=1e-30))
            halves.append((codes[:, :N].view(torch.uint8), scale))
        s["w_codes"] = torch.stack([c for c, _ in halves], 1).contiguous()
        s["w_scales"] = torch.stack([v for _, v in halves], 1).contiguous()
        del halves
        s["start"] = start
        s["cap"] = int((start[1:] - start[:-1]).max())  # a capacity for the plain form's padded products
        s["y"] = torch.zeros(R, N, dtype=_dt(case["out"]), device="cuda")
        return s

    T, H, E, k = (case[n] for n in ("T", "H", "E", "k"))
    R, dt = T * k, _dt(case["dtype"])
    ids, w = _routing(T, E, k, g)
    s["ids"], s["w"] = torch.where(ids < case["held"], ids, torch.full_like(ids, -1)), w
    s["start"], s["rows"], s["pos"] = _order(s["ids"], case["held"])
    if op == "dispatch":
        s["x"] = randn(T, H).to(dt)
        s["xs"] = torch.zeros(R, H, dtype=dt, device="cuda")
        for n, shape in (("start", case["held"] + 1), ("rows", R), ("pos", (T, k))):
            s[n] = torch.zeros(shape, dtype=torch.int32, device="cuda")
        # the most moelora_dispatch_workspace asks for, whatever the token count
        s["ws"] = torch.empty(1024 * (case["held"] + 1), dtype=torch.uint8, device="cuda")
    elif op == "quantize":
        s["x"] = randn(T, H).to(dt)
        s["codes"] = torch.zeros(R, _pitch(H), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros(_pitch(H) // 128, R, device="cuda")
    else:
        s["ys"] = randn(R, H).to(dt)
        if op == "combine_grad":
            s["dout"] = randn(T, H).to(dt)
            s["dys"] = torch.zeros(R, H, dtype=dt, device="cuda")
            s["dw"] = torch.zeros(T, k, device="cuda")
        else:
            s["out"] = torch.zeros(T, H, dtype=dt, device="cuda")
    return s


# --------------------------------------------------------------------- run

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import lora_expert_gemm_amd as lib
    e4m3 = torch.float8_e4m3fn
    op = s["op"]
    if op == "product":
        M, N = s["w_codes"].shape[1], s["N"]
        lib.moelora_fp8_gemm(s["T"] * s["k"], N, s["K"], s["E"],
                             lib.BF16 if s["out"] == BF16 else lib.F32,
                             lib.FP8_SILU_MUL if M == 2 else 0, s["codes"], s["scales"],
                             s["start"], s["w_codes"], s["w_scales"], s["y"])
        return s["y"]
    dt = lib.BF16 if s["dtype"] == BF16 else lib.F32
    if op == "quantize_weights":
        lib.moelora_quantize_weights(s["E"], s["N"], s["K"], dt, s["w"], s["codes"], s["scales"],
                                     s["codes_t"], s["scales_t"])
        return s["codes"].view(e4m3), s["scales"], s["codes_t"].view(e4m3), s["scales_t"]
    T, H, k = s["T"], s["H"], s["k"]
    if op == "dispatch":
        lib.moelora_dispatch(T, H, s["held"], k, dt, s["x"], s["ids"], s["start"], s["rows"],
                             s["pos"], s["xs"], s["ws"], s["ws"].numel())
        return s["start"], s["rows"], s["pos"], s["xs"]
    if op == "dispatch_grad":
        lib.moelora_dispatch_backward(T, H, k, dt, s["ys"], s["pos"], s["out"])
        return s["out"]
    if op == "combine":
        lib.moelora_combine(T, H, k, dt, s["ys"], s["pos"], s["w"], s["out"])
        return s["out"]
    if op == "combine_grad":
        lib.moelora_combine_backward(T, H, k, dt, s["dout"], s["ys"], s["pos"], s["w"], s["dys"],
                                     s["dw"])
        return s["dys"], s["dw"]
    lib.moelora_quantize_rows(T * k, H, dt, s["x"], T, s["rows"], k, s["codes"], s["scales"])
    return s["codes"].view(e4m3), s["scales"]


def _run_plain(s):
    op = s["op"]
    if op == "product":
        return _plain_product(s)
    if op == "quantize_weights":
        N, K = s["N"], s["K"]
        codes, scale = _weight_blocks(s["w"], _pow2_scale)
        flat = codes.view(torch.uint8)
        turned = flat.transpose(1, 2).contiguous()
        e4m3 = torch.float8_e4m3fn
        return (flat[:, :N].contiguous().view(e4m3), scale, turned[:, :K].contiguous().view(e4m3),
                scale.transpose(1, 2).contiguous())
    k = s["k"]
    if op == "dispatch":
        start, rows, pos = _order(s["ids"], s["held"])
        R = rows.numel()
        at = torch.where(rows < R, rows // k, torch.zeros_like(rows)).long()
        xs = torch.where((rows < R)[:, None], s["x"][at], torch.zeros((), dtype=s["x"].dtype,
                                                                       device="cuda"))
        return start, rows, pos, xs
    if op == "quantize":
        rows = s["rows"]
        R = rows.numel()
        ok = rows < R
        codes, scale = _quantize_rows(s["x"][torch.where(ok, rows // k, 0).long()].float())
        codes = torch.where(ok[:, None], codes.view(torch.uint8), 0)
        return codes.view(torch.float8_e4m3fn), torch.where(ok[None], scale, 0.0)
    pos = s["pos"].long()
    ok = pos >= 0
    if op in ("dispatch_grad", "combine"):
        y = torch.where(ok[..., None], s["ys"][pos.clamp(min=0)].float(), 0.0)
        if op == "combine":
            y = y * s["w"][..., None]
        return y.sum(1).to(s["ys"].dtype)
    R = s["ys"].shape[0]
    d = s["dout"].float()[:, None]
    y = torch.where(ok[..., None], s["ys"][pos.clamp(min=0)].float(), 0.0)
    dys = torch.zeros(R + 1, s["ys"].shape[1], dtype=s["ys"].dtype, device="cuda")
    dys[torch.where(ok, pos, R).view(-1)] = (s["w"][..., None] * d).to(dys.dtype).view(R, -1)
    dys[R] = 0
    return dys[:R], (d * y).sum(-1)


def _plain_product(s):
    K, N, E, cap = s["K"], s["N"], s["E"], s["cap"]
    e4m3 = torch.float8_e4m3fn
    R, P = s["codes"].shape
    KB, M = P // 128, s["w_codes"].shape[1]
    x = (s["codes"].view(e4m3).float().view(R, KB, 128) * s["scales"].t()[..., None]).view(R, P)
    per_row = s["w_scales"].repeat_interleave(128, 2)[:, :, :N]  # [E][M][N][KB]
    w = (s["w_codes"].view(e4m3).float().view(E, M, N, KB, 128) * per_row[..., None])
    w = w.view(E, M * N, P)
    start = s["start"].long()
    at = (start[:-1, None] + torch.arange(cap, device="cuda")).clamp(max=R - 1)
    padded = torch.bmm(x[at], w.transpose(1, 2))  # [E][cap][M N], each expert as wide as the fullest
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
    b = 2 if case.get("dtype") == BF16 else 4
    if op == "quantize_weights":
        n = case["E"] * case["N"] * case["K"]
        return {"bytes": n * (b + 2) + 8 * n / 128 ** 2, "flops": 2 * n}
    T, E, k = case["T"], case["E"], case["k"]
    if op == "product":
        R, K = T * k, case["K"]
        width = case["N"] * (2 if case["silu"] else 1)
        hit = E * (1 - (1 - k / E) ** T)  # experts that some token picks
        n = hit * width * K
        out = R * case["N"] * (2 if case["out"] == BF16 else 4)
        return {"bytes": n + n / 4096 + R * K * (1 + 4 / 128) + out, "flops": 2 * R * width * K}
    H = case["H"]
    R, share = T * k, case["held"] / E
    kept = R * share
    if op == "dispatch":
        return {"bytes": T * H * b + kept * H * b + 12 * R, "flops": 0}
    if op == "quantize":
        return {"bytes": T * H * b + kept * (H + H / 32) + 4 * R, "flops": 2 * kept * H}
    n = {"dispatch_grad": kept + T, "combine": kept + T, "combine_grad": 2 * kept + T}[op]
    return {"bytes": n * H * b + 8 * R, "flops": (4 if op == "combine_grad" else 2) * kept * H}


# ------------------------------------------------------------------- exact

def _e4m3_table():
    v = torch.empty(256, dtype=torch.float64)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        a = float("nan") if c & 127 == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = -a if c & 128 else a
    return v.cuda()


def _nearest_e4m3(v):
    """float64 values of at most 448 to the nearest E4M3 value, ties to even."""
    _, ex = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (ex - 4).clamp(min=-9))
    return torch.round(v / step) * step


def _exponent(amax):
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448)).clamp(min=-126)
    e = torch.where(torch.exp2(e - 1) * 448 >= amax, e - 1, e)
    e = torch.where(torch.exp2(e) * 448 < amax, e + 1, e)
    return torch.exp2(e.clamp(min=-126))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f8 = torch.float8_e4m3fn
    if op == "product":
        table, K, N = _e4m3_table(), case["K"], case["N"]
        out = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        rows = table[s["codes"].long()]
        rows *= s["scales"].double().t().repeat_interleave(128, 1)
        start = s["start"].tolist()
        for e in range(case["E"]):
            lo, hi = start[e], start[e + 1]
            if lo == hi:
                continue
            made = []
            for half in range(s["w_codes"].shape[1]):
                w = table[s["w_codes"][e, half].long()]
                by = s["w_scales"][e, half].double().repeat_interleave(128, 0)[:N]
                made.append(rows[lo:hi] @ (w * by.repeat_interleave(128, 1)).t().contiguous())
            out[lo:hi] = made[0] * torch.sigmoid(made[0]) * made[1] if case["silu"] else made[0]
        return out
    if op == "quantize_weights":
        E, N, K = case["E"], case["N"], case["K"]
        got = [torch.zeros(E, N, _pitch(K), dtype=torch.float32, device="cuda"),
               torch.zeros(s["scales"].shape, dtype=torch.float64, device="cuda"),
               torch.zeros(E, K, _pitch(N), dtype=torch.float32, device="cuda"),
               torch.zeros(s["scales_t"].shape, dtype=torch.float64, device="cuda")]
        for e in range(E):
            for b in range(0, N, 128):
                w = torch.zeros(min(128, N - b), _pitch(K), dtype=torch.float64, device="cuda")
                w[:, :K] = s["w"][e, b:b + 128]
                sc = _exponent(w.abs().amax(0).view(-1, 128).amax(1))
                c = _nearest_e4m3(w / sc.repeat_interleave(128))
                got[0][e, b:b + 128] = c
                got[1][e, b // 128] = sc
                got[2][e, :, b:b + c.shape[0]] = c[:, :K].t()
                got[3][e, :, b // 128] = sc
        return got[0].to(f8), got[1], got[2].to(f8), got[3]
    k = case["k"]
    if op in ("dispatch", "quantize"):
        ids, held = s["ids"].view(-1).tolist(), case["held"]
        order = sorted((e, p) for p, e in enumerate(ids) if 0 <= e < held)
        at = torch.tensor([p // k for _, p in order], dtype=torch.long, device="cuda")
        if op == "dispatch":
            xs = torch.zeros(s["xs"].shape, dtype=torch.float64, device="cuda")
            xs[:len(order)] = s["x"][at].double()
            return None, None, None, xs
        H, P = case["H"], _pitch(case["H"])
        codes = torch.zeros(s["codes"].shape, dtype=torch.float32, device="cuda")
        scales = torch.zeros(s["scales"].shape, dtype=torch.float64, device="cuda")
        for b in range(0, P, 128):
            v = torch.zeros(len(order), 128, dtype=torch.float64, device="cuda")
            v[:, :min(128, H - b)] = s["x"][at, b:b + 128]
            sc = _exponent(v.abs().amax(1))
            codes[:len(order), b:b + 128] = _nearest_e4m3(v / sc[:, None])
            scales[b // 128, :len(order)] = sc
        return codes.to(f8), scales
    T, H = case["T"], case["H"]
    total = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    dys = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = torch.nonzero(s["pos"][:, j] >= 0).view(-1)
        p = s["pos"][t, j].long()
        y, w = s["ys"][p].double(), s["w"][t, j].double()
        if op == "combine_grad":
            dys[p] = w[:, None] * s["dout"][t].double()
            dw[t, j] = (y * s["dout"][t].double()).sum(1)
        else:
            total[t] += y * w[:, None] if op == "combine" else y
    return (dys, dw) if op == "combine_grad" else total
