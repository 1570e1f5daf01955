"""Plain 64-bit references of the paged-cache and beam-search operators (loops over
requests, pages and candidates), for the tests."""
from __future__ import annotations

import numpy as np


def ceil_div(a, b):
    return -(-a // b)


def plan(start, count, tokens, ps, n_pages, free, n_free, table, release=False):
    """(table, slots, free, n_free, error) after a plan (or its release)."""
    table, free = table.copy(), free.copy()
    slots = np.full((len(start), tokens), -1, np.int64)
    err, jobs = 0, []
    for b, (s, c) in enumerate(zip(start, count)):
        if s < 0 or c < 0 or (not release and c > tokens) or s + c > table.shape[1] * ps:
            err = err or -3
            continue
        jobs.append((b, s, c, ceil_div(s, ps), ceil_div(s + c, ps)))
    total = sum(j[4] - j[3] for j in jobs)
    if not 0 <= n_free <= n_pages:
        return table, slots, free, n_free, -1
    if (total > n_pages - n_free) if release else (total > n_free):
        return table, slots, free, n_free, -7
    if release:
        top = n_free + total
        for b, s, c, held, need in jobs:
            for j in range(held, need):
                top -= 1
                free[top] = table[b, j]
        return table, slots, free, n_free + total, err
    for b, s, c, held, need in jobs:
        for j in range(held, need):
            n_free -= 1
            table[b, j] = free[n_free]
        for t in range(c):
            page = table[b, (s + t) // ps]
            if 0 <= page < n_pages:
                slots[b, t] = page * ps + (s + t) % ps
            else:
                err = err or -1
    return table, slots, free, n_free, err


def attention(q, k, v):
    """One sequence: q [Hq, D], k, v [Hkv, L, D] (fp64) -> (o, sum p |v| per output, largest sum |q k| scale)."""
    Hq, D = q.shape
    Hkv, L, _ = k.shape
    o, mass, reach = np.zeros((Hq, D)), np.zeros((Hq, D)), 0.0
    if L == 0:
        return o, mass, reach
    for h in range(Hq):
        g = h // (Hq // Hkv)
        s = k[g] @ q[h] / np.sqrt(D)
        p = np.exp(s - s.max())
        p /= p.sum()
        o[h], mass[h] = p @ v[g], p @ np.abs(v[g])
        reach = max(reach, float((np.abs(k[g]) @ np.abs(q[h])).max() / np.sqrt(D)))
    return o, mass, reach


def attention_tol(o, mass, reach, dtype, D, L):
    """Per output, how far a kernel may be from the exact `o`.

    Scores are fp32 sums of D products: each is off by at most (D + 2) 2^-24 sum |q k| scale, which
    moves a weight by that relative amount, as do the weight's own exponential (2^-22) and the sums
    over at most 128 keys, 8 partial sums and ceil(L / 128) folds of three roundings.  bf16 kernels
    round the weights to bf16 (2^-8 at most) before both the products and their normaliser.  Weights and
    normaliser move the quotient by at most twice that of sum p |v|.  The output is rounded once."""
    u = 2.0 ** -24
    w = (D + 2) * u * reach + 2.0 ** -22 + (128 + 8 + 3 * ceil_div(L, 128) + 4) * u
    out = u
    if dtype == "bf16":
        w += 2.0 ** -8
        out = 2.0 ** -8
    w = 2 * w * (1 + w) + 4 * u
    return w * mass + out * (np.abs(o) + w * mass)


def beam_select(logits, scores, beams, n_out, last=None, eos=-1):
    """(parents, tokens, scores) [groups, n_out] from fp64 logits [rows, vocab]."""
    rows, V = logits.shape
    out = []
    with np.errstate(divide="ignore", invalid="ignore"):
        m = logits.max(1, keepdims=True)
        safe = np.where(np.isneginf(m), 0.0, m)
        lse = np.log(np.exp(logits - safe).sum(1, keepdims=True))      # of the logits less the largest
        c = np.where(np.isneginf(m), -np.inf, (logits - safe) - np.where(np.isneginf(m), 0.0, lse)) + scores[:, None]
    c = np.where(np.isneginf(scores)[:, None], -np.inf, c)
    if last is not None:
        for r in np.flatnonzero(last == eos):
            c[r] = -np.inf
            c[r, eos] = scores[r]
    for g in range(rows // beams):
        x = c[g * beams:(g + 1) * beams].reshape(-1)
        if n_out < len(x):
            few = np.flatnonzero(x >= np.partition(x, len(x) - n_out)[len(x) - n_out])
        else:
            few = np.arange(len(x))
        at = few[np.lexsort((few, -x[few]))[:n_out]]
        out.append((at // V + g * beams, at % V, x[at]))
    return tuple(np.stack(z) for z in zip(*out))


def beam_reorder(table, parents, beams, lens, ps, caches, n_pages):
    """(table, caches, error): caches a list of [n_pages, H, ps, D] arrays (K and V of every layer)."""
    table, caches, err = table.copy(), [c.copy() for c in caches], 0
    for g in range(len(parents) // beams):
        rows = range(g * beams, (g + 1) * beams)
        n = lens[rows[0]]
        own = []
        ok = 0 <= n <= table.shape[1] * ps and all(lens[r] == n for r in rows) and all(parents[r] in rows for r in rows)
        if ok and n % ps:
            own = [table[r, n // ps] for r in rows]
            ok = len(set(own)) == beams and all(0 <= p < n_pages for p in own)
        if not ok:
            err = -1
            continue
        c, r = n // ps, n % ps
        table[rows, :c] = table[[parents[i] for i in rows], :c]
        if r:
            for x in caches:
                x[own, :, :r] = x[[own[parents[i] - rows[0]] for i in rows], :, :r]
    return table, caches, err
