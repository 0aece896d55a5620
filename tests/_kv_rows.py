"""Attention over the 8-bit cache in 64 bits, row by row from its definition,
with NaN, missing pages and the scales of pages taken into account, and how far
fp32 sums of fp16 weights may be from it.  Test infrastructure; shares nothing
with the library."""
import math

import numpy as np
import torch

from tests import _kv


def reference(ref, q, cu, lengths, table, scale, causal=True, window=0, heads=None):
    """For the query heads `heads` (all as a rule), [tokens, heads(, dim)] each:
    out and lse, NaN where a row sees one; weight (the probabilities' sum of
    |v|), reach (the largest sum of |q k| scale among a row's keys) and largest
    (the largest probability times its page's scale).  Pages the cache does not
    have are not seen."""
    q = q.double().numpy()
    group = q.shape[1] // ref.scales[0].shape[1]
    heads = list(range(q.shape[1])) if heads is None else heads
    pages_held = len(ref.scales[0])
    shape = (q.shape[0], len(heads))
    out, weight = np.zeros((*shape, q.shape[2])), np.zeros((*shape, q.shape[2]))
    lse, reach, largest = np.full(shape, -math.inf), np.zeros(shape), np.zeros(shape)
    for s, length in enumerate(lengths):
        n = cu[s + 1] - cu[s]
        if n == 0 or length <= 0:
            continue
        ids = np.asarray(table[s][:-(-length // ref.block)], dtype=np.int64)
        held = (ids >= 0) & (ids < pages_held)
        ids = np.where(held, ids, 0)
        k, v = (ref.sequence(half, ids, length) for half in range(2))
        there = np.repeat(held, ref.block)[:length]
        pos, j = np.arange(length - n, length)[:, None], np.arange(length)[None, :]
        seen = np.broadcast_to(there, (n, length))
        if causal:
            seen = seen & (j <= pos)
            if window:
                seen = seen & (j > pos - window)
        for i, h in enumerate(heads):
            kh, vh = k[:, h // group], v[:, h // group]
            unit = np.array([_kv.scale_value(b) for b in ref.scales[1][ids, h // group]])
            unit = np.nan_to_num(np.repeat(unit, ref.block)[:length])
            bad_k, bad_v = np.isnan(kh).any(1), np.isnan(vh)
            kh, vh = np.nan_to_num(kh), np.nan_to_num(vh)
            rows = q[cu[s]:cu[s + 1], h]
            x = np.where(seen, rows @ kh.T * scale, -math.inf)
            top = x.max(1, keepdims=True)
            some = np.isfinite(top)
            p = np.exp(x - np.where(some, top, 0.0))
            total = p.sum(1, keepdims=True)
            p = p / np.where(some, total, 1.0)
            at = slice(cu[s], cu[s + 1])
            out[at, i], weight[at, i] = p @ vh, p @ np.abs(vh)
            with np.errstate(divide="ignore"):
                lse[at, i] = (np.where(some, top, 0.0) + np.log(total))[:, 0]
            reach[at, i] = np.where(seen, np.abs(rows) @ np.abs(kh).T, 0.0).max(1) * abs(scale)
            largest[at, i] = (p * unit).max(1)
            nan_row = (seen & bad_k).any(1)
            out[at, i][(seen.astype(np.float64) @ bad_v > 0) | nan_row[:, None]] = math.nan
            lse[at, i][nan_row] = math.nan
    return out, lse, weight, reach, largest


def bounds(out, weight, reach, largest, keys, dim, bf16):
    """How far an element may be off, and a row's lse.

    Scores, their exponentials and the sums over keys in fp32 as in
    tests/_kv.py.  A probability times its page's scale is rounded to fp16: to
    2^-11 of itself for bf16 queries, 2^-22 as two terms for fp32 ones, and to
    steps of 2^-24 (half of it off) where a row's largest is 2^7 or more: 2^-32
    of that, times 448, for each key.  A bf16 output is off by half a step of
    its 8 bits more."""
    bound, lse = _kv.tolerance(weight, reach, out, keys, dim, False)
    bound = bound + 2.0 ** (-11 if bf16 else -22) * weight
    bound = bound + (keys * 448 * 2.0 ** -32 * largest)[..., None]
    if bf16:
        _, exponent = np.frexp(np.abs(np.nan_to_num(out)) + bound)
        bound = bound + np.ldexp(1.0, exponent - 9)
    return bound, lse


def wide_batch(fp4, cu, lengths, table):
    """A table far wider than the sequences: laid out as for long ones."""
    cu, lengths, table = _kv.batch(fp4, cu, lengths, table)
    return cu, lengths, torch.nn.functional.pad(table, (0, 2 ** 16 - table.shape[1]), value=2 ** 30)


def compare(ref, dev, q, cu, lengths, table, scale=None, heads=None, fp4=None, batch=None,
            **how):
    """The library's rows against the definition's, NaN and -inf where it has
    them; returns out and lse on the CPU."""
    dim, bf16 = q.shape[2], q.dtype == torch.bfloat16
    scale = dim ** -0.5 if scale is None else scale
    batch = _kv.batch(fp4, cu, lengths, table) if batch is None else batch
    got, got_lse = fp4.kv_attention(q.cuda(), dev, *batch, scale=scale, return_lse=True,
                                    check=False, **how)
    want, lse, weight, reach, largest = reference(ref, q, cu, lengths, table, scale, heads=heads,
                                                  **how)
    at = slice(None) if heads is None else heads
    y, y_lse = got.double().cpu().numpy()[:, at], got_lse.double().cpu().numpy()[:, at]
    for a, b, what in ((y, want, "out"), (y_lse, lse, "lse")):
        wrong = np.argwhere((np.isnan(a) != np.isnan(b)) | (np.isinf(a) != np.isinf(b)))
        assert not len(wrong), f"{what}: {len(wrong)} NaN or inf differ, first at {wrong[0]}: " \
                               f"{a[tuple(wrong[0])]} for {b[tuple(wrong[0])]}"
    bound, lse_bound = bounds(want, weight, reach, largest, max(max(lengths), 1), dim, bf16)
    fin = np.isfinite(lse)
    off = np.abs(y_lse - lse)[fin] / (lse_bound + 2.0 ** -23 * np.abs(lse))[fin]
    assert off.size == 0 or off.max() <= 1, f"lse: {off.max()} of the bound"
    off = np.where(np.isnan(want), 0.0, np.abs(y - want) / bound)
    worst = np.unravel_index(off.argmax(), off.shape)
    assert off.max() <= 1, f"{off.max()} of the bound at {worst}: {y[worst]} for {want[worst]}"
    return got.cpu(), got_lse.cpu()
