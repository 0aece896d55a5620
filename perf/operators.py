"""Cases of the 8-bit key/value cache operators: write, read, attention.

The cache is paged.  A page holds ``block`` tokens; per page and kv head it has
``block x d`` E4M3FN codes of keys and as many of values, and one E8M0 byte for
each (value = E4M3(code) * 2^(byte - 127)).  A batch is described by ``cu``
(prefix sums of the new tokens), ``lengths`` (tokens of each sequence, the new
ones included) and ``table`` (page ids): new token i of sequence s sits at
position lengths[s] - (cu[s + 1] - cu[s]) + i.

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
    def case(name, op, seqs, new, length, hkv, group, d, block, dtype="bf16", ragged=True,
             causal=True, window=0, lse=False):
        return {"name": name, "op": op, "seqs": seqs, "new": new, "length": length, "hkv": hkv,
                "group": group, "d": d, "block": block, "dtype": dtype, "ragged": ragged,
                "causal": causal, "window": window, "lse": lse}

    return [
        # one new token for each of a few conversations: a call's latency
        case("write 8 tokens", "write", 8, 1, 1000, 8, 8, 128, 64),
        # chunks of an odd size that start and end inside pages, fp32 keys, small heads
        case("write chunks fp32 d64", "write", 13, 77, 501, 4, 4, 64, 16, dtype="fp32"),
        # whole prompts
        case("write prompts", "write", 8, 4096, 4096, 8, 8, 128, 64),
        # a few short conversations read back for another consumer, in fp32
        case("read short fp32 d64", "read", 5, 77, 77, 4, 4, 64, 16, dtype="fp32"),
        # a batch of long ones read back
        case("read prompts", "read", 16, 4096, 4096, 8, 8, 128, 64),
        # one conversation, one token: latency
        case("attend 1 x 1000", "attend", 1, 1, 1000, 8, 8, 128, 64, ragged=False),
        # a batch of decoding conversations, shared kv heads
        case("attend 64 x 8192", "attend", 64, 1, 8192, 8, 8, 128, 64),
        # one very long conversation
        case("attend 1 x 200001", "attend", 1, 1, 200001, 8, 8, 128, 128, ragged=False, lse=True),
        # every query head with a kv head of its own, fp32 queries, small heads and pages
        case("attend 16 x 2048 fp32 d64", "attend", 16, 1, 2048, 16, 1, 64, 16, dtype="fp32"),
        # a few drafted tokens each, a sliding window, wide heads
        case("attend 24 x 5 window d256", "attend", 24, 5, 4096, 4, 4, 256, 32, window=1024),
        # chunks of prompts against what is cached already
        case("attend chunks 4 x 1024", "attend", 4, 1024, 6000, 8, 8, 128, 64),
        # a whole prompt
        case("attend prompt 4096", "attend", 1, 4096, 4096, 8, 4, 128, 64, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend"])
    d = rng.choice([64, 128, 128, 128, 192, 256])
    block = rng.choice([16, 32, 64, 128])
    hkv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 4, 5, 7, 8, 16])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    causal, window = True, 0
    if op == "attend":
        if rng.random() < 0.65:  # decoding, a few drafted tokens among it
            new = rng.choice([1, 1, 1, 2, 3, 6])
            seqs = _log(rng, 1, 96)
            length = _log(rng, 7, 30000)
            window = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
            most = 4e8
        else:  # chunks and prompts
            new = _log(rng, 17, 3000)
            seqs = _log(rng, 1, 8)
            length = new + rng.choice([0, _log(rng, 16, 6000)])
            causal = rng.random() < 0.8
            window = rng.choice([0, 0, _log(rng, 16, 2048)]) if causal else 0
            most = 2e8
        while seqs * length * hkv * d > most and seqs > 1:
            seqs = seqs // 2
        while new > 16 and seqs * new * length * hkv * group * d > 3e11:
            new, length = new // 2, max(new // 2, length // 2)
    else:
        new = rng.choice([1, _log(rng, 2, 4096)])
        seqs = _log(rng, 1, 256 if new == 1 else 16)
        length = new if op == "read" else new + rng.choice([0, _log(rng, 1, 3000)])
    return {"op": op, "seqs": seqs, "new": new, "length": length, "hkv": hkv, "group": group,
            "d": d, "block": block, "dtype": dtype, "ragged": rng.random() < 0.7,
            "causal": causal, "window": window, "lse": rng.random() < 0.3}


def _sizes(case):
    """New tokens and lengths (with them) of each sequence, from the case alone."""
    new, length = [], []
    for s in range(case["seqs"]):
        f = 0.5 + (s + 1) * GOLDEN % 1.0 if case["ragged"] else 1.0
        n = case["new"] if case["new"] == 1 else max(1, int(case["new"] * f))
        old = int((case["length"] - case["new"]) * f)
        new.append(n)
        length.append(n + old)
    return new, length


def _pairs(case):
    """Visible (query token, cached token) pairs."""
    total = 0
    for n, length in zip(*_sizes(case)):
        if not case["causal"]:
            total += n * length
            continue
        last = torch.arange(length - n, length, dtype=torch.int64) + 1
        total += int((torch.clamp(last, max=case["window"]) if case["window"] else last).sum())
    return total


def work(case):
    new, length = _sizes(case)
    row = case["hkv"] * case["d"]
    wide = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "attend":
        seen = sum(min(l, n + case["window"] - 1) if case["window"] else l
                   for n, l in zip(new, length))
        return {"bytes": 2 * seen * row + 2 * sum(new) * row * case["group"] * wide,
                "flops": 4 * _pairs(case) * row * case["group"]}
    moved = 2 * sum(new) * row * (1 + wide)
    return {"bytes": moved, "flops": 2 * sum(new) * row}


# ---- inputs ----------------------------------------------------------------
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    new, length = _sizes(case)
    seqs, hkv, d, block = case["seqs"], case["hkv"], case["d"], case["block"]
    width = max(-(-n // block) for n in length)  # pages of the longest sequence
    used = [-(-n // block) for n in length]
    pages = sum(used) + 3  # a few stay free
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(seqs, width, dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(used):
        table[s, :n] = order[at:at + n]
        at += n
    cu = torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32).to(dev)
    lengths = torch.tensor(length, dtype=torch.int32, device=dev)

    def half(outliers):
        """Codes and scales of one half of the cache: normal values, a few wide channels."""
        codes = torch.empty(pages, hkv, block, d, dtype=torch.uint8, device=dev)
        step = max(1, (1 << 27) // (hkv * block * d))
        for p in range(0, pages, step):
            x = torch.randn(codes[p:p + step].shape, generator=g, device=dev) * 50
            if outliers:
                x[..., 3::32] *= 3
            codes[p:p + step] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        scales = torch.randint(120, 123, (pages, hkv), generator=g, device=dev).to(torch.uint8)
        return codes, scales

    k_codes, k_scales = half(True)
    v_codes, v_scales = half(False)
    state = {"case": case, "k_codes": k_codes, "k_scales": k_scales, "v_codes": v_codes,
             "v_scales": v_scales, "cu": cu, "lengths": lengths, "table": table,
             "tokens": sum(new), "most_new": max(new)}
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "write":
        # keys and values as they come out of one projection: slices of its rows
        x = torch.randn(sum(new), 2 * hkv, d, generator=g, device=dev)
        x[:, :hkv, 3::32] *= 6
        x = x.to(dtype)
        state["k"], state["v"] = x[:, :hkv], x[:, hkv:]
    if case["op"] == "attend":
        q = torch.randn(sum(new), hkv * case["group"], d, generator=g, device=dev)
        state["q"] = (q * 1.5).to(dtype)
    return state


# ---- the plain forms, in 32 bits -------------------------------------------
def _e4m3(y):
    """The nearest E4M3 values of |y| <= 448, ties to the even one."""
    _, exponent = torch.frexp(y)
    step = torch.clamp(exponent - 1, min=-6) - 3
    unit = torch.exp2(step.to(y.dtype))
    return torch.round(y / unit) * unit


def _value(codes):
    """The E4M3 values of codes, from their fields."""
    c = codes.to(torch.int32)
    e, m = (c >> 3) & 15, c & 7
    v = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).float()), m * 2.0 ** -9)
    return torch.where(c >= 128, -v, v)


def _code(value):
    """The codes of E4M3 values (exact: nothing is rounded here)."""
    return value.to(torch.float8_e4m3fn).view(torch.uint8)


def _scale(byte):
    return torch.exp2(byte.to(torch.float32) - 127)


def _slots(state):
    """Each new token's sequence, position, page and slot."""
    t = torch.arange(state["tokens"], device="cuda")
    cu, lengths, block = state["cu"].long(), state["lengths"].long(), state["case"]["block"]
    s = torch.searchsorted(cu, t, right=True) - 1
    pos = lengths[s] - cu[s + 1] + t
    return s, pos, state["table"].long()[s, pos // block], pos % block


def _write_half(codes, scales, x, state):
    s, pos, page, slot = _slots(state)
    block = state["case"]["block"]
    x = x.to(torch.float32)
    pages, hkv = scales.shape
    amax = torch.zeros(pages, hkv, device=x.device)
    amax.scatter_reduce_(0, page[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
    m, e = torch.frexp(amax)
    byte = torch.where(amax > 0, torch.clamp(e + 118 + (m > 0.875), min=0), 0)
    # live tokens of a page: those before its first new one
    first = torch.full((pages,), block, device=x.device).scatter_reduce_(0, page, slot, "amin")
    touched = first < block
    old = scales.to(torch.int64)
    byte = torch.where((first > 0)[:, None], torch.maximum(byte, old), byte)
    byte = torch.where(touched[:, None], byte, old)
    # a grown scale moves the live codes down
    grown = torch.nonzero(touched & (first > 0) & (byte > old).any(1)).flatten()
    down = torch.exp2((old - byte)[grown].float())[:, :, None, None]
    live = torch.arange(block, device=x.device)[None, :] < first[grown, None]
    moved = _code(_e4m3(_value(codes[grown]) * down))
    codes[grown] = torch.where(live[:, None, :, None], moved, codes[grown])
    codes[page, :, slot] = _code(_e4m3(x * torch.exp2(127 - byte[page].float())[:, :, None]))
    scales.copy_(byte)


def _gather(codes, scales, table):
    """Values of whole sequences [seqs, hkv, width * block, d], in 32 bits."""
    t = table.long()
    x = _value(codes[t]) * _scale(scales[t])[..., None, None]  # [S, P, H, B, D]
    x = x.transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _attend(state):
    case, q = state["case"], state["q"]
    hkv, group, d = case["hkv"], case["group"], case["d"]
    k = _gather(state["k_codes"], state["k_scales"], state["table"])
    v = _gather(state["v_codes"], state["v_scales"], state["table"])
    seqs, most = case["seqs"], state["most_new"]
    cu, lengths = state["cu"].long(), state["lengths"].long()
    t = torch.arange(state["tokens"], device=q.device)
    s = torch.searchsorted(cu, t, right=True) - 1
    rows = torch.zeros(seqs, most, hkv, group, d, device=q.device)
    rows[s, t - cu[s]] = q.to(torch.float32).view(-1, hkv, group, d)
    rows = rows.permute(0, 2, 3, 1, 4).reshape(seqs, hkv, group * most, d)
    score = torch.matmul(rows, k.transpose(2, 3).contiguous()) * d ** -0.5
    score = score.view(seqs, hkv, group, most, -1)
    j = torch.arange(k.shape[2], device=q.device)
    if case["causal"]:
        pos = (lengths - (cu[1:] - cu[:-1]))[:, None] + torch.arange(most, device=q.device)
        seen = j <= pos[..., None]
        if case["window"]:
            seen &= j > pos[..., None] - case["window"]
    else:
        seen = (j < lengths[:, None])[:, None].expand(-1, most, -1)
    seen = seen & (j < lengths[:, None])[:, None]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = torch.where((j < lengths[:, None])[:, None, :, None], v, torch.zeros_like(v))
    out = torch.matmul(p.view(seqs, hkv, group * most, -1), v).view(seqs, hkv, group, most, d)
    out = out / torch.where(total > 0, total, torch.ones_like(total))
    out = out.permute(0, 3, 1, 2, 4)[s, t - cu[s]].reshape(-1, hkv * group, d).to(q.dtype)
    if not case["lse"]:
        return {"out": out}
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2)[s, t - cu[s]]
    return {"out": out, "lse": lse.reshape(-1, hkv * group)}


def _cache_out(state):
    return {"k": state["k_codes"].view(torch.float8_e4m3fn), "k_scales": state["k_scales"],
            "v": state["v_codes"].view(torch.float8_e4m3fn), "v_scales": state["v_scales"]}


def _run_plain(state):
    op = state["case"]["op"]
    if op == "write":
        _write_half(state["k_codes"], state["k_scales"], state["k"], state)
        _write_half(state["v_codes"], state["v_scales"], state["v"], state)
        return _cache_out(state)
    if op == "read":
        _, _, page, slot = _slots(state)
        dtype = DTYPES[state["case"]["dtype"]]
        k = _value(state["k_codes"][page, :, slot]) * _scale(state["k_scales"][page])[..., None]
        v = _value(state["v_codes"][page, :, slot]) * _scale(state["v_scales"][page])[..., None]
        return {"k": k.to(dtype), "v": v.to(dtype)}
    return _attend(state)


# ---- one pass --------------------------------------------------------------
def run(state):
    if not own:
        return _run_plain(state)
    import mxfp4_block_amax_amd as fp4

    case = state["case"]
    cache = fp4.KVCache(state["k_codes"], state["k_scales"], state["v_codes"], state["v_scales"])
    cu, lengths, table = state["cu"], state["lengths"], state["table"]
    if case["op"] == "write":
        fp4.kv_cache_write(cache, state["k"], state["v"], cu, lengths, table, check=False)
        return _cache_out(state)
    if case["op"] == "read":
        k, v = fp4.kv_cache_read(cache, cu, lengths, table, state["tokens"],
                                 out_dtype=DTYPES[case["dtype"]], check=False)
        return {"k": k, "v": v}
    got = fp4.kv_attention(state["q"], cache, cu, lengths, table, causal=case["causal"],
                           window=case["window"], return_lse=case["lse"], check=False)
    return {"out": got[0], "lse": got[1]} if case["lse"] else {"out": got}


# ---- the definition, in 64 bits --------------------------------------------
def _table64():
    """The 256 E4M3FN values."""
    values = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.ldexp(8 + m, e - 10) if e else math.ldexp(m, -9)
        if c & 127 == 127:
            v = math.nan
        values.append(-v if c >= 128 else v)
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def _nearest64(y, table):
    """The nearest E4M3 values by search among all of them, ties to the even code."""
    grid = table[:127]
    y_abs = y.abs()
    hi = torch.searchsorted(grid, y_abs.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - y_abs, y_abs - grid[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(grid[pick], y)


def _exact_write(state, table):
    case, block = state["case"], state["case"]["block"]
    cu, lengths, pages = state["cu"].tolist(), state["lengths"].tolist(), state["table"].tolist()
    outs = {}
    for name in ("k", "v"):
        values = table[state[name + "_codes"].long()]
        scales = state[name + "_scales"].to(torch.int64).cpu()
        x = state[name].to(torch.float64)
        for s in range(case["seqs"]):
            start = lengths[s] - (cu[s + 1] - cu[s])
            pos = start
            while pos < lengths[s]:
                end = min(lengths[s], (pos // block + 1) * block)
                page, slot = pages[s][pos // block], pos % block
                part = x[cu[s] + pos - start:cu[s] + end - start].transpose(0, 1)  # [H, n, D]
                for h, top in enumerate(part.abs().amax((1, 2)).tolist()):
                    byte = 0
                    if top > 0:
                        byte = max(0, math.ceil(math.log2(top / 448)) + 126)
                        while math.ldexp(448.0, byte - 127) < top:
                            byte += 1
                    if slot > 0:
                        before = int(scales[page, h])
                        if byte > before:
                            moved = values[page, h, :slot] * 2.0 ** (before - byte)
                            values[page, h, :slot] = _nearest64(moved, table)
                        byte = max(byte, before)
                    scales[page, h] = byte
                    values[page, h, slot:slot + end - pos] = _nearest64(
                        part[h] * 2.0 ** (127 - byte), table)
                pos = end
        outs[name], outs[name + "_scales"] = values, scales.to(torch.uint8).cuda()
    return outs


def _sequence64(codes, scales, pages, n, table):
    """One sequence's values [hkv, n, d]."""
    p = pages[:-(-n // codes.shape[2])].long()
    x = table[codes[p].long()] * torch.exp2(scales[p].double() - 127)[..., None, None]
    return x.transpose(0, 1).reshape(codes.shape[1], -1, codes.shape[3])[:, :n]


def exact(case, seed):
    state = prepare(case, seed)
    table = _table64()
    if case["op"] == "write":
        return _exact_write(state, table)
    parts = {"k": [], "v": [], "out": [], "lse": []}
    cu, lengths = state["cu"].tolist(), state["lengths"].tolist()
    for s in range(case["seqs"]):
        n, length = cu[s + 1] - cu[s], lengths[s]
        k = _sequence64(state["k_codes"], state["k_scales"], state["table"][s], length, table)
        v = _sequence64(state["v_codes"], state["v_scales"], state["table"][s], length, table)
        if case["op"] == "read":
            parts["k"].append(k[:, length - n:].transpose(0, 1))
            parts["v"].append(v[:, length - n:].transpose(0, 1))
            continue
        q = state["q"][cu[s]:cu[s + 1]].double().transpose(0, 1)  # [Hq, n, D]
        pos = torch.arange(length - n, length, device="cuda")[:, None]
        j = torch.arange(length, device="cuda")[None, :]
        hidden = torch.zeros(n, length, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden = j > pos
            if case["window"]:
                hidden |= j <= pos - case["window"]
        out, lse = [], []
        for h in range(case["hkv"]):
            qh = q[h * case["group"]:(h + 1) * case["group"]].reshape(-1, case["d"])
            a = (qh @ k[h].t().contiguous()).view(case["group"], n, length) / math.sqrt(case["d"])
            a.masked_fill_(hidden, -math.inf)
            z = torch.logsumexp(a, -1)
            out.append((torch.exp(a - z[..., None]).view(-1, length) @ v[h]).view(
                case["group"], n, case["d"]))
            lse.append(z)
        parts["out"].append(torch.cat(out).transpose(0, 1))
        parts["lse"].append(torch.cat(lse).transpose(0, 1))
    if case["op"] == "read":
        return {"k": torch.cat(parts["k"]), "v": torch.cat(parts["v"])}
    got = {"out": torch.cat(parts["out"])}
    if case["lse"]:
        got["lse"] = torch.cat(parts["lse"])
    return got
