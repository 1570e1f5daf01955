"""Plain 64-bit references of the chunk attention, the log probabilities and the sharing of pages, for the tests."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24


def ceil_div(a, b):
    return -(-a // b)


def chunk_attention(q, k, v, start):
    """One sequence: q [T, Hq, D], k, v [Hkv, start + T, D] (fp64) -> (o, sum p |v|, largest sum |q k| scale)."""
    T, Hq, D = q.shape
    Hkv, L, _ = k.shape
    group = Hq // Hkv
    qh = q.permute(1, 0, 2).reshape(Hkv, group * T, D)
    s = torch.einsum("gtd,gld->gtl", qh, k) * D ** -0.5
    reach = torch.einsum("gtd,gld->gtl", qh.abs(), k.abs()) * D ** -0.5
    t = torch.arange(T, device=q.device).repeat(group)
    hidden = torch.arange(L, device=q.device)[None, :] > (start + t)[:, None]
    s = s.masked_fill(hidden[None], float("-inf"))
    p = torch.softmax(s, 2)

    def rows(x):
        return x.reshape(Hkv, group, T, D).permute(2, 0, 1, 3).reshape(T, Hq, D)
    return rows(p @ v), rows(p @ v.abs()), float(reach.masked_fill(hidden[None], 0.0).max())


def chunk_tol(o, mass, reach, dtype, D, L):
    """Per output, how far a kernel may be from the exact `o`.

    Scores are fp32 sums of D products: each is off by at most (D + 2) 2^-24 sum |q k| scale, which moves a weight by
    that relative amount, as do the weight's own exponential (2^-22) and the sums: at most 128 keys of a chunk, the 8
    partial sums of its threads, three roundings for each chunk of 64 keys or more that is folded, and three for each of
    at most 304 joined pieces (no more than there are chunks).  bf16 kernels round the weights to bf16 (2^-8 at most)
    before the products.  Weights and normaliser move the quotient by at most twice that of sum
    p |v|.  The output is rounded once."""
    chunks = ceil_div(L, 64)
    w = (D + 2) * U * reach + 2.0 ** -22 + (128 + 8 + 3 * chunks + 3 * min(304, chunks) + 4) * U
    out = U
    if dtype == torch.bfloat16:
        w += 2.0 ** -8
        out = 2.0 ** -8
    w = 2 * w * (1 + w) + 4 * U
    return w * mass + out * (o.abs() + w * mass)


def token_logprobs(z, token, n_top):
    """One row of fp32 logits (numpy) -> (log probability or None, entropy, ids, their log probabilities), in fp64."""
    z = np.asarray(z, np.float64)
    m = z.max()
    if np.isneginf(m):
        lp, h = np.full(len(z), -np.inf), 0.0
    else:
        lp = (z - m) - np.log(np.exp(z - m).sum())
        p = np.exp(lp)
        h = float(-(p[p > 0] * lp[p > 0]).sum())
    ids = np.lexsort((np.arange(len(z)), -z))[:n_top]
    return (None if token is None else lp[token]), h, ids, lp[ids]


def logprob_tol(lp, z, V):
    """How far a log probability may be off: x = z - max is rounded once (2^-24 |x|, for the token and as an exponent);
    an exponential is off by 2^-22 relative at most beside that of its exponent, which is at most 2^-24 times 104 where
    the exponential is not 0 in fp32.  The sums are held in fp32, all terms of one sign, and are off by 2^-24 relative for
    each addition or product on the way of a term: a lane takes 16 logits of a segment of 512 in 5, and moves and adds
    its sums in 4 a segment, of which it has ceil(V / 2048) + 1 at most (4 warps a row); 5 additions over a warp; 4 in
    each of 9 joins at most, of which only those of two parts with terms round: 2, 5 and 9 up to 3, 18 and more segments.
    That is at most 22 below 1024 logits, V / 512 + 38 below 9216 and V / 512 + 54 from there: below V / 256 + 36."""
    rel = (104 + 4 + ceil_div(V, 256) + 32) * U
    return rel + U * np.abs(z - np.max(z)) + U * np.abs(lp)


def entropy_tol(h, V):
    """The sums s and t = sum e x are off by the relative amounts of logprob_tol (all terms of each have one sign), t / s
    by twice that and a rounding per product; |t / s| <= h and log s <= h."""
    rel = (104 + 6 + ceil_div(V, 256) + 32) * U
    return rel * (1 + 2 * abs(h)) + U * abs(h) + V * 2.0 ** -126


def fork(src, dst, lens, ps, n_pages, refs, free, n_free, table, caches):
    """(refs, table, caches, n_free, error): caches a list of [n_pages, H, ps, D] arrays."""
    refs, table, caches = refs.copy(), table.copy(), [c.copy() for c in caches]
    rows, stride = table.shape
    err, jobs = 0, []
    for i, (s, d, n) in enumerate(zip(src, dst, lens)):
        if not (0 <= s < rows and 0 <= d < rows) or list(dst).count(d) > 1 or d in list(src):
            err = err or -1
        elif not 0 <= n <= stride * ps:
            err = err or -3
        else:
            jobs.append((s, d, n // ps, n % ps))
    fresh = sum(1 for j in jobs if j[3])
    if not 0 <= n_free <= n_pages:
        return refs, table, caches, n_free, -1
    if fresh > n_free:
        return refs, table, caches, n_free, -7
    for s, d, full, rest in jobs:
        for j in range(full):
            table[d, j] = p = table[s, j]
            if 0 <= p < n_pages:
                refs[p] += 1
            else:
                err = err or -1
        if rest:
            n_free -= 1
            table[d, full] = to = free[n_free]
            at = table[s, full]
            if not (0 <= to < n_pages and 0 <= at < n_pages):
                err = err or -1
                continue
            for c in caches:
                c[to, :, :rest] = c[at, :, :rest]
    return refs, table, caches, n_free, err


def free_rows(rows_list, lens, ps, n_pages, refs, free, n_free, table):
    """(refs, free, n_free, error)."""
    refs, free = refs.copy(), free.copy()
    rows, stride = table.shape
    err, entries = 0, []
    for r, n in zip(rows_list, lens):
        if not 0 <= r < rows or list(rows_list).count(r) > 1:
            err = err or -1
        elif not 0 <= n <= stride * ps:
            err = err or -3
        else:
            for j in range(ceil_div(n, ps)):
                p = table[r, j]
                if 0 <= p < n_pages:
                    entries.append(p)
                else:
                    err = err or -1
    back = []
    last = {p: e for e, p in enumerate(entries)}
    for e, p in enumerate(entries):
        if last[p] == e and entries.count(p) >= refs[p] + 1:
            back.append(p)
    if not 0 <= n_free <= n_pages:
        return refs, free, n_free, -1
    if n_free + len(back) > n_pages:
        return refs, free, n_free, -7
    for p in set(entries):
        d = entries.count(p)
        if d > refs[p] + 1:
            err = err or -1
        refs[p] = max(0, refs[p] - d)
    for k, p in enumerate(back):
        free[n_free + len(back) - 1 - k] = p
    return refs, free, n_free + len(back), err
