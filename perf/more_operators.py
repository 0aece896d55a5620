"""Cases of what a decoding layer does with four-bit weights and few tokens:
the product of activations that keep their precision with an FP4 weight, a
router and the gated products of the experts that it chooses, and the norm and
position rotation of queries and keys ahead of the cache.

A weight [rows, K] is E2M1 codes (two a byte, the even element in the low
nibble) and a scale for 32 (MXFP4, E8M0) or 16 (NVFP4, E4M3, times one fp32
scale of the tensor) consecutive values; ``packed`` is the same bytes in MFMA
operand order.

``run`` with ``own`` false computes each operator in elementary torch
operations in 32 bits; with ``own`` true it calls the framework.  ``exact`` has
the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
GOLDEN = 0.6180339887498949


# ---- cases -----------------------------------------------------------------
def listed():
    def linear(name, m, n, k, fmt="mxfp4", dtype="bf16", packed=False):
        return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "fmt": fmt, "dtype": dtype,
                "packed": packed}

    def route(name, tokens, hidden, experts, top, dtype="bf16", router="bf16", renormalize=True):
        return {"name": name, "op": "route", "tokens": tokens, "hidden": hidden,
                "experts": experts, "top": top, "dtype": dtype, "router": router,
                "renormalize": renormalize}

    def experts(name, tokens, hidden, inner, experts, top, fmt="mxfp4", dtype="bf16", pad=0):
        return {"name": name, "op": "experts", "tokens": tokens, "hidden": hidden, "inner": inner,
                "experts": experts, "top": top, "fmt": fmt, "dtype": dtype, "pad": pad}

    def rotate(name, seqs, new, length, hq, hk, d, dtype="bf16", rotary=None, norm=True,
               interleaved=False, ragged=True):
        return {"name": name, "op": "rotate", "seqs": seqs, "new": new, "length": length,
                "hq": hq, "hk": hk, "d": d, "dtype": dtype, "rotary": rotary or d, "norm": norm,
                "interleaved": interleaved, "ragged": ragged}

    return [
        # one token through a small projection: a call's latency
        linear("linear 1 x 512 x 2048", 1, 512, 2048),
        # one token through a square projection, the weight as the W4A4 prefill keeps it
        linear("linear 1 x 8192 x 8192 packed", 1, 8192, 8192, packed=True),
        # a few drafted tokens in fp32, nothing a multiple of a tile
        linear("linear 5 x 5001 x 4112 nvfp4 fp32", 5, 5001, 4112, fmt="nvfp4", dtype="fp32"),
        # a small batch through the projection back from a wide inner layer
        linear("linear 16 x 8192 x 28672 nvfp4", 16, 8192, 28672, fmt="nvfp4"),
        # a batch of decoding conversations through the projection into that layer
        linear("linear 64 x 28672 x 8192 packed", 64, 28672, 8192, packed=True),
        # one token's experts
        route("route 1 x 2048 of 64", 1, 2048, 64, 4),
        # a batch's experts, the router's weight kept in fp32
        route("route 64 x 4096 of 256", 64, 4096, 256, 8, router="fp32"),
        # one token through its experts
        experts("experts 1 x 2048 x 768 of 64", 1, 2048, 768, 64, 4),
        # a few tokens in fp32, two rows of the batch empty, no size a multiple of a tile
        experts("experts 7 x 1040 x 496 nvfp4 fp32", 7, 1040, 496, 20, 3, fmt="nvfp4",
                dtype="fp32", pad=2),
        # a batch of decoding conversations: most experts of the layer are read
        experts("experts 16 x 4096 x 1536 of 128", 16, 4096, 1536, 128, 8),
        # one token's queries and keys
        rotate("rotate 1 x 64 + 8 heads", 1, 1, 1000, 64, 8, 128, ragged=False),
        # prompts, at positions that go on from what is cached
        rotate("rotate 4 x 2048", 4, 2048, 9000, 32, 8, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "route", "experts", "experts", "rotate"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    fmt = rng.choice(["mxfp4", "mxfp4", "nvfp4"])
    if op == "linear":
        packed = rng.random() < 0.4
        step = 512 if packed else 32 if fmt == "mxfp4" else 16
        m = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 17, 64), _log(rng, 65, 130)])
        k = max(1, _log(rng, 256, 28672) // step) * step
        n = _log(rng, 16, 32768)
        while m * n * k > 64 * 8192 * 28672 or n * k > 8192 * 28672:
            n = n // 2
        return {"op": op, "m": m, "n": n, "k": k, "fmt": fmt, "dtype": dtype, "packed": packed}
    if op == "route":
        experts = _log(rng, 4, 512)
        return {"op": op, "tokens": rng.choice([1, _log(rng, 2, 128)]),
                "hidden": _log(rng, 32, 1024) * 8, "experts": experts,
                "top": min(experts, rng.choice([1, 2, 4, 6, 8])), "dtype": dtype,
                "router": rng.choice(["bf16", "fp32"]), "renormalize": rng.random() < 0.7}
    if op == "experts":
        step = 32 if fmt == "mxfp4" else 16
        experts = _log(rng, 4, 256)
        top = min(experts, rng.choice([1, 2, 4, 6, 8]))
        tokens = rng.choice([1, _log(rng, 2, 16), _log(rng, 17, 64)])
        hidden = max(1, _log(rng, 256, 8192) // step) * step
        inner = max(1, _log(rng, 128, 4096) // step) * step
        while experts * hidden * inner > 128 * 4096 * 1536:
            inner = max(step, inner // 2 // step * step)
            hidden = max(step, hidden // 2 // step * step)
        while tokens > 1 and tokens * top * hidden * inner > 16 * 8 * 4096 * 1536:
            tokens = tokens // 2
        return {"op": op, "tokens": tokens, "hidden": hidden, "inner": inner, "experts": experts,
                "top": top, "fmt": fmt, "dtype": dtype,
                "pad": rng.choice([0, 0, tokens // 3])}
    d = rng.choice([64, 128, 128, 192, 256])
    new = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 17, 4096)])
    hk = rng.choice([1, 2, 4, 8, 16])
    hq = hk * rng.choice([1, 2, 4, 5, 8])
    seqs = _log(rng, 1, 64)
    while seqs > 1 and seqs * new * (hq + hk) * d > 4 * 2048 * 40 * 128:
        seqs = seqs // 2
    while new > 1 and seqs * new * (hq + hk) * d > 4 * 2048 * 40 * 128:
        new = new // 2
    return {"op": op, "seqs": seqs, "new": new,
            "length": new + rng.choice([0, _log(rng, 1, 1000000)]), "hq": hq, "hk": hk, "d": d,
            "dtype": dtype, "rotary": rng.choice([d, d, d // 2]), "norm": rng.random() < 0.7,
            "interleaved": rng.random() < 0.3, "ragged": rng.random() < 0.7}


def _sizes(case):
    """New tokens and lengths (with them) of each sequence, from the case alone."""
    new, length = [], []
    for s in range(case["seqs"]):
        f = 0.5 + (s + 1) * GOLDEN % 1.0 if case["ragged"] else 1.0
        n = case["new"] if case["new"] == 1 else max(1, int(case["new"] * f))
        new.append(n)
        length.append(n + int((case["length"] - case["new"]) * f))
    return new, length


def _weight_bytes(case, rows, k):
    return rows * k // 2 + rows * k // (32 if case["fmt"] == "mxfp4" else 16)


def work(case):
    wide = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": _weight_bytes(case, n, k) + m * (n + k) * wide, "flops": 2 * m * n * k}
    if case["op"] == "route":
        t, h, e, top = case["tokens"], case["hidden"], case["experts"], case["top"]
        return {"bytes": t * h * wide + e * h * (4 if case["router"] == "fp32" else 2)
                + t * top * 8, "flops": 2 * t * h * e}
    if case["op"] == "experts":
        t, h, i, top = case["tokens"] - case["pad"], case["hidden"], case["inner"], case["top"]
        # the experts that some token goes to, on average over even choices
        read = case["experts"] * (1 - (1 - top / case["experts"]) ** t)
        return {"bytes": int(read * _weight_bytes(case, 3 * h, i))
                + case["tokens"] * (2 * h * wide + top * 8), "flops": 6 * t * top * h * i}
    row = sum(_sizes(case)[0]) * (case["hq"] + case["hk"]) * case["d"]
    return {"bytes": 2 * row * wide, "flops": row * (8 if case["norm"] else 4)}


# ---- inputs ----------------------------------------------------------------
def _codes(shape, g):
    """E2M1 codes as a normal weight gives them: its magnitudes, scaled so that a
    block's largest is near 6, fall on 0, 0.5, .. 6 with these weights of 128."""
    nibble = []
    for code, count in enumerate((13, 24, 21, 18, 25, 15, 10, 2)):
        nibble += [code] * count
    nibble = torch.tensor(nibble + [8 + c for c in nibble], dtype=torch.uint8, device="cuda")
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    flat, step = out.view(-1), 1 << 26
    for at in range(0, flat.numel(), step):
        part = flat[at:at + step]
        r = torch.randint(0, 65536, part.shape, generator=g, device="cuda", dtype=torch.int32)
        part.copy_(nibble[r & 255] | nibble[r >> 8] << 4)
    return out


def _weight(fmt, shape, g):
    """Codes, scales and tensor scales (one for each leading index) of weights
    [.., rows, K] whose values are some K ** -0.5."""
    k = shape[-1]
    codes = _codes((*shape[:-1], k // 2), g)
    if fmt == "mxfp4":
        at = 126 + round(math.log2(0.6 * k ** -0.5))
        scales = torch.randint(at, at + 3, (*shape[:-1], k // 32), generator=g, device="cuda",
                               dtype=torch.uint8)
        return codes, scales, None
    # E4M3 codes of 16 .. 30 times a tensor scale
    scales = torch.randint(0x58, 0x5F, (*shape[:-1], k // 16), generator=g, device="cuda",
                           dtype=torch.uint8)
    lead = math.prod(shape[:-2])
    s_g = torch.rand(lead, generator=g, device="cuda") * 0.2 + 0.9
    return codes, scales, s_g * (0.02 * k ** -0.5)


def _pack(fmt, codes, scales):
    """The same bytes in MFMA operand order (row tiles of 32, K steps of 64)."""
    n, half = codes.shape
    rt, ks = -(-n // 32), half // 32
    c = torch.zeros(rt * 32, half, dtype=torch.uint8, device="cuda")
    c[:n] = codes
    c = c.view(rt, 32, ks, 2, 16).permute(0, 2, 3, 1, 4).reshape(-1)
    s = torch.full((rt * 32, scales.shape[1]), 127 if fmt == "mxfp4" else 0, dtype=torch.uint8,
                   device="cuda")
    s[:n] = scales
    if fmt == "mxfp4":
        s = s.view(rt, 32, ks // 8, 8, 2).permute(0, 2, 4, 1, 3)
    else:
        s = s.view(rt, 32, ks // 8, 8, 2, 2).permute(0, 2, 4, 1, 3, 5)
    return torch.cat([c, s.reshape(-1)])


def _activations(shape, g, dtype):
    """Normal values, a few channels several times as wide."""
    x = torch.randn(shape, generator=g, device="cuda")
    x[..., 5::97] *= 6
    return x.to(DTYPES[dtype])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"case": case}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        state["x"] = _activations((m, k), g, case["dtype"])
        state["weight"] = _weight(case["fmt"], (n, k), g)
        if case["packed"]:
            state["packed"] = _pack(case["fmt"], *state["weight"][:2])
    elif case["op"] == "route":
        t, h, e = case["tokens"], case["hidden"], case["experts"]
        state["x"] = _activations((t, h), g, case["dtype"])
        router = torch.randn(e, h, generator=g, device="cuda") * h ** -0.5
        state["router"] = router.to(DTYPES[case["router"]])
    elif case["op"] == "experts":
        t, h, i, e = case["tokens"], case["hidden"], case["inner"], case["experts"]
        state["x"] = _activations((t, h), g, case["dtype"])
        logit, chosen = torch.rand(t, e, generator=g, device="cuda").topk(case["top"], dim=1)
        chosen[t - case["pad"]:] = -1  # rows of the batch that hold no token
        state["experts"] = chosen.to(torch.int32)
        state["weights"] = torch.softmax(logit * 4, 1)
        state["up"] = _weight(case["fmt"], (e, 2 * i, h), g)
        state["down"] = _weight(case["fmt"], (e, h, i), g)
    else:
        new, length = _sizes(case)
        tokens, heads, d = sum(new), case["hq"] + case["hk"], case["d"]
        state["cu"] = torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
        state["lengths"] = torch.tensor(length, dtype=torch.int32).cuda()
        state["tokens"] = tokens
        # queries and keys as they come out of one projection: slices of its rows
        x = torch.randn(tokens, heads + case["hk"], d, generator=g, device="cuda")
        x[:, :, 3::32] *= 6
        x = x.to(DTYPES[case["dtype"]])
        state["q"], state["k"] = x[:, :case["hq"]], x[:, case["hq"]:heads]
        state["frequencies"] = 500000.0 ** -(
            torch.arange(0, case["rotary"], 2, dtype=torch.float64, device="cuda")
            / case["rotary"])
        if case["norm"]:
            w = 1 + 0.3 * torch.randn(2, d, generator=g, device="cuda")
            state["q_weight"], state["k_weight"] = w.to(DTYPES[case["dtype"]])
    return state


# ---- the plain forms, in 32 bits -------------------------------------------
def _elements(codes):
    """The E2M1 values of packed codes, from their fields."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    e, m = (c >> 1 & 3).float(), (c & 1).float()
    v = torch.where(e > 0, (2 + m) * torch.exp2(e - 2), m * 0.5)
    return torch.where(c >= 8, -v, v)


def _scale_values(fmt, scales):
    s = scales.to(torch.int32)
    if fmt == "mxfp4":
        return torch.exp2((s - 127).float())
    e, m = s >> 3 & 15, s & 7
    v = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).float()), m * 2.0 ** -9)
    return torch.where(s >= 128, -v, v)


def _widen(fmt, codes, scales):
    """A weight's values in 32 bits, but for its tensor scale."""
    v = _elements(codes)
    s = _scale_values(fmt, scales)
    return (v.view(*s.shape, -1) * s[..., None]).view(v.shape)


def _linear(state):
    fmt = state["case"]["fmt"]
    codes, scales, s_g = state["weight"]
    c = state["x"].float() @ _widen(fmt, codes, scales).t()
    return {"c": (c if s_g is None else c * s_g).to(state["x"].dtype)}


def _route(state):
    case = state["case"]
    # choices next to a border must not hang on the order of a sum: 64 bits
    logit = state["x"].double() @ state["router"].double().t()
    rows = torch.arange(case["tokens"], device="cuda")
    left, chosen, value = logit.clone(), [], []
    for _ in range(case["top"]):
        top = left.amax(1)
        at = (left == top[:, None]).to(torch.uint8).argmax(1)  # the first of equal ones
        left[rows, at] = -math.inf
        chosen.append(at)
        value.append(top)
    value = torch.stack(value, 1)
    p = torch.exp(value - value[:, :1])
    if case["renormalize"]:
        p = p / p.sum(1, keepdim=True)
    else:
        p = p / torch.exp(logit - value[:, :1]).sum(1, keepdim=True)
    return {"experts": torch.stack(chosen, 1).to(torch.int32), "weights": p.float()}


def _expert(fmt, x, up, down, inner):
    """One expert's gated product of rows x; up and down as codes, scales, tensor scale."""
    h = x @ _widen(fmt, *up[:2]).t()
    if up[2] is not None:
        h = h * up[2]
    gate, h = h[..., :inner], h[..., inner:]
    y = (gate / (1 + torch.exp(-gate)) * h) @ _widen(fmt, *down[:2]).t()
    return y if down[2] is None else y * down[2]


def _experts(state):
    case, x = state["case"], state["x"].float()
    chosen, weights = state["experts"].long(), state["weights"]
    out = torch.zeros_like(x)
    if case["tokens"] * case["top"] < case["experts"]:
        for t in range(case["tokens"]):
            for j in range(case["top"]):
                e = chosen[t, j:j + 1].clamp(min=0)
                up, down = ([None if w is None else w[e][0] for w in state[n]]
                            for n in ("up", "down"))
                y = _expert(case["fmt"], x[t:t + 1], up, down, case["inner"])
                out[t] += torch.where(chosen[t, j] >= 0, weights[t, j] * y[0], 0.0)
    else:
        for e in range(case["experts"]):
            share = torch.where(chosen == e, weights, 0.0).sum(1, keepdim=True)
            up, down = ([None if w is None else w[e] for w in state[n]] for n in ("up", "down"))
            y = _expert(case["fmt"], x, up, down, case["inner"])
            out += torch.where((chosen == e).any(1, keepdim=True), share * y, 0.0)
    return {"out": out.to(state["x"].dtype)}


EPS = 1e-6


def _rotate_rows(x, weight, c, s, case):
    x = x.float()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    r = case["rotary"]
    y = x.clone()
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * c - b * s, a * s + b * c
    return y


def _rotate(state):
    case, dtype = state["case"], state["q"].dtype
    cu, lengths = state["cu"].long(), state["lengths"].long()
    t = torch.arange(state["tokens"], device="cuda")
    s = torch.searchsorted(cu, t, right=True) - 1
    pos = lengths[s] - cu[s + 1] + t
    angle = pos.double()[:, None, None] * state["frequencies"]
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    return {n: _rotate_rows(state[n], state.get(n + "_weight"), c, s, case).to(dtype)
            for n in ("q", "k")}


# ---- one pass --------------------------------------------------------------
def run(state):
    case = state["case"]
    if not own:
        return {"linear": _linear, "route": _route, "experts": _experts,
                "rotate": _rotate}[case["op"]](state)
    import mxfp4_block_amax_amd as fp4

    if case["op"] == "linear":
        fmt = fp4.MXFP4 if case["fmt"] == "mxfp4" else fp4.NVFP4
        codes, scales, s_g = state["weight"]
        if case["packed"]:
            return {"c": fp4.linear_w4_packed(fmt, state["x"], state["packed"], case["n"], s_g)}
        return {"c": fp4.linear_w4(fmt, state["x"], codes, scales, s_g)}
    if case["op"] == "route":
        chosen, weights = fp4.moe_route(state["x"], state["router"], case["top"],
                                        renormalize=case["renormalize"])
        return {"experts": chosen, "weights": weights}
    if case["op"] == "experts":
        fmt = fp4.MXFP4 if case["fmt"] == "mxfp4" else fp4.NVFP4
        return {"out": fp4.moe_experts(fmt, state["x"], state["experts"], state["weights"],
                                       state["up"], state["down"], check=False)}
    q, k = fp4.norm_rotate(state["q"], state["k"], state["cu"], state["lengths"],
                           state["frequencies"], state.get("q_weight"), state.get("k_weight"),
                           eps=EPS, interleaved=case["interleaved"], check=False)
    return {"q": q, "k": k}


# ---- the definition, in 64 bits --------------------------------------------
def _weight64(fmt, codes, scales, s_g):
    """A weight's values by tables of all codes."""
    grid = [0, .5, 1, 1.5, 2, 3, 4, 6]
    e2m1 = torch.tensor(grid + [-v for v in grid], dtype=torch.float64, device="cuda")
    if fmt == "mxfp4":
        table = [2.0 ** (b - 127) for b in range(255)] + [math.nan]
    else:
        table = [math.ldexp(b & 7, -9) if b < 8 else math.ldexp(8 + (b & 7), (b >> 3) - 10)
                 for b in range(127)] + [math.nan]
        table += [-v for v in table]
    block = 32 if fmt == "mxfp4" else 16
    w = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device="cuda")
    w[:, 0::2], w[:, 1::2] = e2m1[(codes & 15).int()], e2m1[(codes >> 4).int()]
    table = torch.tensor(table, dtype=torch.float64, device="cuda")
    w *= table[scales.int()].repeat_interleave(block, 1)
    return w if s_g is None else w * s_g.double()


def _exact_route(state):
    case = state["case"]
    logit = torch.matmul(state["x"].double(), state["router"].double().t().contiguous())
    order = torch.sort(logit, dim=1, descending=True, stable=True)
    chosen, value = order.indices[:, :case["top"]], order.values[:, :case["top"]]
    over = value if case["renormalize"] else logit
    weights = torch.exp(value - torch.logsumexp(over, 1, keepdim=True))
    return {"experts": chosen.to(torch.int32), "weights": weights}


def _exact_experts(state):
    case, x = state["case"], state["x"].double()
    out = torch.zeros_like(x)
    chosen = state["experts"].tolist()
    tokens = {}
    for t, row in enumerate(chosen):
        for j, e in enumerate(row):
            if e >= 0:
                tokens.setdefault(e, []).append((t, j))
    for e, at in sorted(tokens.items()):
        (up, down) = (_weight64(case["fmt"], w[0][e], w[1][e], None if w[2] is None else w[2][e])
                      for w in (state["up"], state["down"]))
        rows = torch.tensor([t for t, _ in at], device="cuda")
        slots = torch.tensor([j for _, j in at], device="cuda")
        h = x[rows] @ up.t()
        gate, h = h[:, :case["inner"]], h[:, case["inner"]:]
        y = (h * gate * torch.sigmoid(gate)) @ down.t()
        out.index_put_((rows,), y * state["weights"][rows, slots].double()[:, None],
                       accumulate=True)
    return {"out": out}


def _exact_rotate(state):
    case, outs = state["case"], {}
    cu, lengths = state["cu"].tolist(), state["lengths"].tolist()
    pos = torch.cat([torch.arange(n - (b - a), n) for a, b, n in zip(cu, cu[1:], lengths)])
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       pos.cuda().double()[:, None] * state["frequencies"])[:, None]
    r = case["rotary"]
    for name in ("q", "k"):
        x = state[name].double()
        if case["norm"]:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
            x = x * state[name + "_weight"].double()
        pairs = x[..., :r].unflatten(-1, (-1, 2) if case["interleaved"] else (2, -1))
        a, b = pairs.unbind(-1 if case["interleaved"] else -2)
        z = torch.complex(a, b) * turn
        z = torch.stack([z.real, z.imag], -1 if case["interleaved"] else -2).flatten(-2)
        outs[name] = torch.cat([z, x[..., r:]], -1)
    return outs


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "linear":
        codes, scales, s_g = state["weight"]
        step = max(1, (1 << 26) // case["k"])
        parts = [state["x"].double() @ _weight64(case["fmt"], codes[i:i + step],
                                                 scales[i:i + step], s_g).t()
                 for i in range(0, case["n"], step)]
        return {"c": torch.cat(parts, 1)}
    return {"route": _exact_route, "experts": _exact_experts,
            "rotate": _exact_rotate}[case["op"]](state)
