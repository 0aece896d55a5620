"""The 8-bit key/value cache in 64 bits on the CPU, from its definition: one
token, page and head at a time, with E4M3 rounding as a search among all its
values.  Test infrastructure; shares nothing with the library."""
import math

import numpy as np
import torch


def e4m3_values():
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = math.ldexp(8 + m, e - 10) if e else math.ldexp(m, -9)
        a = math.nan if c & 127 == 127 else a
        v[c] = -a if c >= 128 else a
    return v


VALUES = e4m3_values()
GRID = VALUES[:127]


def e4m3_codes(y):
    """Nearest codes of float64 values (|y| <= 448 or NaN), ties to even."""
    y = np.asarray(y, dtype=np.float64)
    a = np.where(np.isnan(y), 0.0, np.abs(y))
    assert (a <= 448).all()
    hi = np.clip(np.searchsorted(GRID, a), 1, 126)
    lo = hi - 1
    up, down = GRID[hi] - a, a - GRID[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.isnan(y), 127, pick + np.where(np.signbit(y), 128, 0))
    return code.astype(np.uint8)


def scale_byte(amax):
    if amax == 0:
        return 0
    e = -127
    while math.ldexp(448.0, e) < amax:
        e += 1
    return e + 127


def scale_value(byte):
    return math.nan if byte == 255 else math.ldexp(1.0, int(byte) - 127)


class Cache:
    """k and v as numpy code and scale arrays, written token range by range."""

    def __init__(self, pages, heads, block, dim, seed=0):
        g = np.random.default_rng(seed)
        self.block = block
        # what a page held before is arbitrary, NaN codes and scales included
        self.codes = [g.integers(0, 256, (pages, heads, block, dim)).astype(np.uint8)
                      for _ in range(2)]
        self.scales = [g.integers(0, 256, (pages, heads)).astype(np.uint8) for _ in range(2)]

    def write(self, kv, cu, lengths, table):
        for half, x in enumerate(kv):
            x = np.asarray(x, dtype=np.float64)
            codes, scales = self.codes[half], self.scales[half]
            for s, length in enumerate(lengths):
                n = cu[s + 1] - cu[s]
                p = length - n
                while p < length:
                    end = min(length, (p // self.block + 1) * self.block)
                    page, slot = table[s][p // self.block], p % self.block
                    for h in range(x.shape[1]):
                        rows = x[cu[s] + p - (length - n):cu[s] + end - (length - n), h]
                        finite = np.isfinite(rows)
                        byte = scale_byte(np.abs(rows[finite]).max(initial=0.0))
                        if slot:
                            old = int(scales[page, h])
                            byte = max(byte, old)
                            moved = VALUES[codes[page, h, :slot]] * 2.0 ** (old - byte)
                            if byte > old:
                                codes[page, h, :slot] = e4m3_codes(moved)
                        scales[page, h] = byte
                        y = np.where(finite, rows, math.nan) * 2.0 ** (127 - byte)
                        codes[page, h, slot:slot + end - p] = e4m3_codes(y)
                    p = end

    def sequence(self, half, pages, length):
        """[length, heads, dim] of one sequence."""
        p = np.asarray(pages[:-(-length // self.block)], dtype=np.int64)
        scale = np.array([scale_value(b) for b in range(256)])[self.scales[half][p]]
        x = VALUES[self.codes[half][p]] * scale[..., None, None]
        return x.transpose(0, 2, 1, 3).reshape(-1, x.shape[1], x.shape[3])[:length]

    def device(self, fp4):
        put = [torch.from_numpy(a.copy()).cuda()
               for a in (self.codes[0], self.scales[0], self.codes[1], self.scales[1])]
        return fp4.KVCache(*put)


def attention(cache, q, cu, lengths, table, scale, causal=True, window=0):
    """out, lse, and what the tolerances need, all [tokens, heads(, dim)]:
    weight (the probabilities' sum of |v|) and reach (the largest sum of
    |q k| scale over a row's keys) in float64."""
    q = np.asarray(q, dtype=np.float64)
    out, weight = np.zeros_like(q), np.zeros_like(q)
    lse, reach = np.full(q.shape[:2], -math.inf), np.zeros(q.shape[:2])
    for s, length in enumerate(lengths):
        n = cu[s + 1] - cu[s]
        if n == 0 or length <= 0:
            continue
        k, v = (cache.sequence(half, table[s], length) for half in range(2))
        group = q.shape[1] // k.shape[1]
        for h in range(q.shape[1]):
            kh, vh = k[:, h // group], v[:, h // group]
            rows = q[cu[s]:cu[s + 1], h]
            score = rows @ kh.T * scale
            pos = np.arange(length - n, length)[:, None]
            j = np.arange(length)[None, :]
            seen = (j <= pos) if causal else np.ones_like(score, dtype=bool)
            if window:
                seen &= j > pos - window
            for i in range(n):
                at = np.nonzero(seen[i])[0]
                if not len(at):
                    continue
                x = score[i, at]
                top = x.max()
                p = np.exp(x - top)
                t = cu[s] + i
                out[t, h] = p @ vh[at] / p.sum()
                weight[t, h] = p @ np.abs(vh[at]) / p.sum()
                lse[t, h] = top + math.log(p.sum())
                reach[t, h] = (np.abs(rows[i]) @ np.abs(kh[at]).T).max() * abs(scale)
    return out, lse, weight, reach


def tolerance(weight, reach, out, keys, dim, bf16):
    """How far an fp32 softmax may be off, per element.

    A score is an fp32 sum of dim products (dim 2^-24 of the sum of their
    magnitudes, as much again for the products split over operands), scaled and
    turned into a base-2 exponent (4 roundings of at most reach); that error is
    the probability's relative one, once above and once below the fraction.
    The sums over keys add keys 2^-24.  With bf16 queries a probability is
    rounded to bf16 (2^-9) and so is the output."""
    u = 2.0 ** -24
    score = (2 * dim + 8) * u * reach
    rel = 2 * score + 2 * (keys + 16) * u
    bound = rel[..., None] * weight
    if bf16:
        bound = bound + 2.0 ** -9 * weight + 2.0 ** -9 * (np.abs(out) + bound)
    return bound + 1e-30, score + (keys + 16) * u


def batch(fp4, cu, lengths, table):
    return (torch.tensor(cu, dtype=torch.int32, device="cuda"),
            torch.tensor(lengths, dtype=torch.int32, device="cuda"),
            torch.tensor(table, dtype=torch.int32, device="cuda"))


def layout(new, before, block, spare=2, seed=0):
    """(cu, lengths, table, pages) of sequences with `new` tokens after
    `before`, their pages in random order; entries past a sequence's length are
    ids no cache has."""
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    lengths = [n + b for n, b in zip(new, before)]
    used = [-(-n // block) for n in lengths]
    pages = sum(used) + spare
    order = np.random.default_rng(seed).permutation(pages)
    width = max(max(used), 1)
    table, at = np.full((len(new), width), 2 ** 30, dtype=np.int64), 0
    for s, n in enumerate(used):
        table[s, :n] = order[at:at + n]
        at += n
    return cu, lengths, table.tolist(), pages
