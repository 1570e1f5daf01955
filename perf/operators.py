"""Cases of the paged-cache and beam-search operators: inputs, plain forms, the library's calls and 64-bit results.

Five operators that a serving loop runs together: llama_paged_plan / llama_paged_release (block tables and slot maps
from request lengths), llama_paged_store (prefilled rows into pages), llama_paged_attention (one new token per sequence
over the pages), llama_beam_select (the best continuations of each request's beams) and llama_beam_reorder (block
tables and unfilled last pages follow the chosen parents).

Sizes: the 8B block (32 / 8 heads of 128, vocabulary 128,256, batch 32 at 1000 cached positions), the 70B block
(64 / 8 heads, batch 16 at 8192 positions) and the tiny fp32 block (4 / 2 heads of 64) of this repository, and
generic page sizes, batches and lengths.
"""
import math

import numpy as np
import torch

own = False

VOCAB = 128256
NEG = float("-inf")


def listed():
    return [
        # one decode step of 64 running requests: each may need one fresh page
        {"name": "plan_step", "op": "plan", "batch": 64, "tokens": 1, "page": 16, "held": 4096, "least": 1},
        # a large admission: 256 prompts of 1 to 4096 tokens get all their pages and slots at once
        {"name": "plan_prompts", "op": "plan", "batch": 256, "tokens": 4096, "page": 16, "held": 0, "least": 1},
        # one prefill chunk of 8 requests goes to their pages (8B block, ragged ends)
        {"name": "store_chunk", "op": "store", "batch": 8, "tokens": 512, "page": 16, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "least": 100},
        # 32 prefilled prompts of up to 2048 tokens go to their pages
        {"name": "store_prompts", "op": "store", "batch": 32, "tokens": 2048, "page": 64, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "least": 1024},
        # the tiny fp32 block after 16 prefilled and up to 4 decoded tokens: the smallest call, latency alone
        {"name": "attention_tiny_f32", "op": "attention", "batch": 2, "heads": 4, "kv_heads": 2, "dim": 64,
         "dtype": "f32", "page": 16, "longest": 20, "least": 17},
        # the 8B decode step of the benchmark (batch 32 near 1000 cached positions) on 16-token pages
        {"name": "attention_8b_b32", "op": "attention", "batch": 32, "heads": 32, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "page": 16, "longest": 1057, "least": 945},
        # the 70B decode step (batch 16 near 8192 cached positions)
        {"name": "attention_70b_b16", "op": "attention", "batch": 16, "heads": 64, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "page": 64, "longest": 8193, "least": 7937},
        # one long conversation alone: the split over the cache's length carries all the parallel work
        {"name": "attention_long_b1", "op": "attention", "batch": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "page": 128, "longest": 131072, "least": 131072},
        # the first step of one request's beam search: one live beam of four
        {"name": "select_first", "op": "select", "groups": 1, "beams": 4, "vocab": VOCAB, "n_out": 4, "first": True,
         "ended": 0},
        # a step of 32 requests with 8 beams, one of them ended, twice as many candidates as beams
        {"name": "select_batch", "op": "select", "groups": 32, "beams": 8, "vocab": VOCAB, "n_out": 16,
         "first": False, "ended": 1},
        # one request's four beams on one layer
        {"name": "reorder_one", "op": "reorder", "groups": 1, "beams": 4, "layers": 1, "page": 16, "kv_heads": 8,
         "dim": 128, "dtype": "bf16", "shared": 1000, "len": 1023},
        # 8 requests of four beams through all 32 layers of the 8B stack
        {"name": "reorder_8b", "op": "reorder", "groups": 8, "beams": 4, "layers": 32, "page": 32, "kv_heads": 8,
         "dim": 128, "dtype": "bf16", "shared": 480, "len": 636},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "release", "store", "attention", "attention", "attention", "select", "reorder"])
    page = rng.choice([16, 32, 64, 128])
    if op in ("plan", "release"):
        batch, tokens = _log(rng, 1, 512), _log(rng, 1, 4096)
        tokens = min(tokens, (1 << 20) // batch)
        return {"op": op, "batch": batch, "tokens": tokens, "page": page, "held": rng.choice([0, _log(rng, 1, 4096)]),
                "least": rng.choice([0, 1, tokens])}
    if op == "store":
        bf16 = rng.random() < 0.8
        kv_heads = rng.choice([1, 2, 4, 8])
        batch, tokens = _log(rng, 1, 64), _log(rng, 1, 4096)
        tokens = max(1, min(tokens, (1 << 19) // (batch * kv_heads * (1 if bf16 else 2))))
        return {"op": op, "batch": batch, "tokens": tokens, "page": page, "kv_heads": kv_heads,
                "dim": 128 if bf16 else rng.choice([32, 64, 128]), "dtype": "bf16" if bf16 else "f32",
                "least": rng.randint(0, tokens)}
    if op == "attention":
        bf16 = rng.random() < 0.8
        kv_heads = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 8] if bf16 else [1, 2, 3, 4])
        longest, batch = _log(rng, 1, 65536), _log(rng, 1, 128)
        most = (1 << 20) // kv_heads if bf16 else (1 << 16) // kv_heads
        batch = max(1, min(batch, most // longest))
        longest = min(longest, most)
        return {"op": op, "batch": batch, "heads": kv_heads * group, "kv_heads": kv_heads,
                "dim": 128 if bf16 else rng.choice([32, 64, 128]), "dtype": "bf16" if bf16 else "f32", "page": page,
                "longest": longest, "least": rng.choice([0, 1, max(1, longest // 2), longest])}
    if op == "select":
        beams, vocab = rng.randint(1, 16), _log(rng, 1000, VOCAB)
        groups = min(_log(rng, 1, 32), 256 // beams)
        return {"op": op, "groups": groups, "beams": beams, "vocab": vocab,
                "n_out": min(vocab, rng.choice([beams, 2 * beams])), "first": rng.random() < 0.2,
                "ended": rng.choice([0, 0, rng.randint(0, beams - 1)])}
    shared, new = _log(rng, 1, 2000), _log(rng, 1, 200)
    return {"op": "reorder", "groups": _log(rng, 1, 8), "beams": rng.randint(2, 8), "layers": _log(rng, 1, 32),
            "page": page, "kv_heads": rng.choice([1, 2, 4, 8]), "dim": 128, "dtype": "bf16", "shared": shared,
            "len": shared + new}


# ----------------------------------------------------------------------------- inputs

def _spread(least, most, n, gen):
    """n whole numbers spread evenly over least .. most, in an order from the seed."""
    v = least + (torch.arange(n, device="cuda") * (most - least)) // max(1, n - 1) if n > 1 else \
        torch.full((1,), most, device="cuda")
    return v[torch.randperm(n, generator=gen, device="cuda")].to(torch.int32)


def _np_spread(least, most, n):
    return [least + i * (most - least) // (n - 1) for i in range(n)] if n > 1 else [most]


def _ceil(a, b):
    return -(-a // b)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _tables(need, columns, n_pages, gen):
    """A block table [len(need), columns] with need[b] distinct pages in random order, -1 behind them."""
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    first = torch.cumsum(need, 0) - need
    col = torch.arange(columns, device="cuda")[None, :]
    at = (first[:, None] + col).clamp(max=n_pages - 1)
    return torch.where(col < need[:, None], perm[at], torch.full_like(perm[at], -1)).contiguous()


def _pages(case, n_pages, gen, layers=None):
    shape = (n_pages, case["kv_heads"], case["page"], case["dim"])
    if layers is not None:
        shape = (layers,) + shape
    return tuple(torch.randn(shape, generator=gen, device="cuda", dtype=_dtype(case)) for _ in range(2))


def _prepare_plan(case, gen):
    B, T, ps = case["batch"], case["tokens"], case["page"]
    start = torch.randint(0, case["held"] + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    count = _spread(case["least"], T, B, gen)
    columns = _ceil(case["held"] + T, ps) + 1
    n_pages = B * columns + 37
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    held = (start + ps - 1) // ps
    need = (start + count + ps - 1) // ps
    full = held if case["op"] == "plan" else need
    col = torch.arange(columns, device="cuda")[None, :]
    first = (torch.cumsum(full, 0) - full)[:, None]
    table = torch.where(col < full[:, None], order[(first + col).clamp(max=n_pages - 1)],
                        torch.full((1, 1), -1, device="cuda", dtype=torch.int32)).contiguous()
    used = int(full.sum())
    free = torch.cat([order[used:], torch.full((used,), -1, device="cuda", dtype=torch.int32)]).contiguous()
    pool = torch.tensor([n_pages - used, 0], dtype=torch.int32, device="cuda")
    return {"start": start, "count": count, "table": table, "free": free, "pool": pool,
            "pool_out": torch.zeros(2, dtype=torch.int32, device="cuda"), "n_pages": n_pages,
            "slots": torch.empty(B, T, dtype=torch.int32, device="cuda")}


def _prepare_store(case, gen):
    B, T, ps = case["batch"], case["tokens"], case["page"]
    count = _spread(case["least"], T, B, gen)
    n_pages = B * _ceil(T, ps) + 5
    table = _tables(torch.full((B,), _ceil(T, ps), device="cuda"), _ceil(T, ps), n_pages, gen)
    t = torch.arange(T, device="cuda")
    slots = table[:, t // ps] * ps + t % ps
    slots = torch.where(t[None, :] < count[:, None], slots, torch.full_like(slots, -1)).to(torch.int32).contiguous()
    shape = (B, case["kv_heads"], T, case["dim"])
    k, v = (torch.randn(shape, generator=gen, device="cuda", dtype=_dtype(case)) for _ in range(2))
    pk, pv = _pages(case, n_pages, gen)
    return {"k": k, "v": v, "slots": slots, "pk": pk, "pv": pv}


def _prepare_attention(case, gen):
    B, ps = case["batch"], case["page"]
    lens = _spread(case["least"], case["longest"], B, gen)
    need = (lens + ps - 1) // ps
    columns = _ceil(case["longest"], ps) + 1
    n_pages = int(need.sum()) + 3
    pk, pv = _pages(case, n_pages, gen)
    q = torch.randn(B, case["heads"], case["dim"], generator=gen, device="cuda", dtype=_dtype(case))
    return {"q": q, "pk": pk, "pv": pv, "table": _tables(need, columns, n_pages, gen), "lens": lens,
            "longest": case["longest"], "o": torch.empty_like(q)}


def _prepare_select(case, gen):
    G, K, V, n = case["groups"], case["beams"], case["vocab"], case["n_out"]
    logits = torch.randn(G * K, V, generator=gen, device="cuda") * 3.0
    scores = -20.0 * torch.rand(G, K, generator=gen, device="cuda")
    if case["first"]:
        scores[:, 0] = 0.0
        scores[:, 1:] = NEG
    eos = V - 1
    last = torch.randint(0, V - 1, (G, K), generator=gen, device="cuda", dtype=torch.int32)
    rank = torch.rand(G, K, generator=gen, device="cuda").argsort(1)
    last = torch.where(rank < case["ended"], torch.full_like(last, eos), last)
    return {"logits": logits, "scores": scores.reshape(-1).contiguous(), "last": last.reshape(-1).contiguous(),
            "eos": eos, "groups": G, "beams": K, "n_out": n,
            "parents": torch.empty(G, n, dtype=torch.int32, device="cuda"),
            "tokens": torch.empty(G, n, dtype=torch.int32, device="cuda"),
            "best": torch.empty(G, n, dtype=torch.float32, device="cuda")}


def _prepare_reorder(case, gen):
    G, K, ps, total = case["groups"], case["beams"], case["page"], case["len"]
    full = case["shared"] // ps                  # pages that all beams of a request share
    columns = _ceil(total, ps) + 1
    priv = columns - full
    n_pages = G * (full + K * priv) + 3
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    shared = perm[: G * full].view(G, 1, full).expand(G, K, full)
    private = perm[G * full: G * full + G * K * priv].view(G, K, priv)
    table = torch.cat([shared, private], 2).reshape(G * K, columns).contiguous()
    parents = torch.randint(0, K, (G, K), generator=gen, device="cuda", dtype=torch.int32)
    parents = (parents + K * torch.arange(G, device="cuda", dtype=torch.int32)[:, None]).reshape(-1).contiguous()
    pk, pv = _pages(case, n_pages, gen, case["layers"])
    return {"table": table, "parents": parents, "pk": pk, "pv": pv, "beams": K,
            "lens": torch.full((G * K,), total, dtype=torch.int32, device="cuda")}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    make = {"plan": _prepare_plan, "release": _prepare_plan, "store": _prepare_store, "attention": _prepare_attention,
            "select": _prepare_select, "reorder": _prepare_reorder}[op]
    state = make(case, gen)
    state["op"], state["page"] = op, case.get("page", 0)
    state["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:
        import dense_decoder_block_gb300 as ddb
        state["ddb"] = ddb
        if op in ("store", "attention"):
            state["cache"] = ddb.PagedCache(state["pk"], state["pv"])
        if op == "reorder":
            state["cache"] = ddb.PagedCacheList([ddb.PagedCache(k, v) for k, v in zip(state["pk"], state["pv"])])
        need = 0
        if op == "attention":
            need = ddb.llama_paged_attention_workspace_bytes(case["batch"], case["heads"], case["kv_heads"],
                                                             case["dim"], case["longest"])
        if op == "select":
            need = ddb.llama_beam_select_workspace_bytes(case["groups"], case["beams"], case["vocab"], case["n_out"])
        state["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return state


# ----------------------------------------------------------------------------- the library's calls

def _run_own(s):
    ddb, op = s["ddb"], s["op"]
    if op == "plan":
        ddb.llama_paged_plan(s["start"], s["count"], s["page"], s["n_pages"], s["free"], s["pool"], s["table"],
                             s["slots"], pool_out=s["pool_out"], err_dev=s["err"])
        return {"table": s["table"], "slots": s["slots"], "free": s["pool_out"][:1]}
    if op == "release":
        ddb.llama_paged_release(s["start"], s["count"], s["page"], s["n_pages"], s["free"], s["pool"], s["table"],
                                pool_out=s["pool_out"], err_dev=s["err"])
        return {"pages": s["free"], "free": s["pool_out"][:1]}
    if op == "store":
        ddb.llama_paged_store(s["k"], s["v"], s["slots"], s["cache"], err_dev=s["err"])
        return {"k": s["pk"], "v": s["pv"]}
    if op == "attention":
        ddb.llama_paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["longest"], s["o"], s["ws"],
                                  err_dev=s["err"])
        return s["o"]
    if op == "select":
        ddb.llama_beam_select(s["logits"], s["scores"], s["beams"], s["n_out"], s["parents"], s["tokens"], s["best"],
                              s["ws"], last=s["last"], eos=s["eos"])
        return {"parents": s["parents"], "tokens": s["tokens"], "scores": s["best"]}
    ddb.llama_beam_reorder(s["parents"], s["beams"], s["lens"], s["table"], s["cache"], err_dev=s["err"])
    return {"table": s["table"], "k": s["pk"], "v": s["pv"]}


# ----------------------------------------------------------------------------- plain forms

def _plain_plan(s):
    ps, start, count, table = s["page"], s["start"], s["count"], s["table"]
    held, need = (start + ps - 1) // ps, (start + count + ps - 1) // ps
    fresh = need - held
    off = torch.cumsum(fresh, 0) - fresh
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    at = s["pool"][0] - 1 - (off[:, None] + col - held[:, None])
    new = (col >= held[:, None]) & (col < need[:, None])
    table.copy_(torch.where(new, s["free"][at.clamp(0, s["n_pages"] - 1)], table))
    t = torch.arange(s["slots"].shape[1], device="cuda")[None, :]
    pos = start[:, None] + t
    page = torch.gather(table, 1, (pos // ps).clamp(max=table.shape[1] - 1))
    s["slots"].copy_(torch.where(t < count[:, None], page * ps + pos % ps, torch.full_like(page, -1)))
    s["pool_out"][0] = s["pool"][0] - fresh.sum()
    return {"table": table, "slots": s["slots"], "free": s["pool_out"][:1]}


def _plain_release(s):
    ps, start, count, table, free = s["page"], s["start"], s["count"], s["table"], s["free"]
    held, need = (start + ps - 1) // ps, (start + count + ps - 1) // ps
    fresh = need - held
    off = torch.cumsum(fresh, 0) - fresh
    total = fresh.sum()
    # the stack from its old top: the last page of the last request first
    at = torch.arange(free.shape[0], device="cuda") - s["pool"][0]
    rank = (total - 1 - at).clamp(min=0)
    b = (torch.searchsorted(off + fresh, rank, right=True)).clamp(max=len(start) - 1)
    page = table[b, (held[b] + rank - off[b]).clamp(0, table.shape[1] - 1)]
    free.copy_(torch.where((at >= 0) & (at < total), page, free))
    s["pool_out"][0] = s["pool"][0] + total
    return {"pages": free, "free": s["pool_out"][:1]}


def _plain_store(s):
    B, H, T, D = s["k"].shape
    n, ps = s["pk"].shape[0], s["page"]
    # the token that each slot takes (the one place behind the slots: tokens without one)
    token = torch.full((n * ps + 1,), -1, dtype=torch.int64, device="cuda")
    token[torch.where(s["slots"] >= 0, s["slots"], torch.full_like(s["slots"], n * ps)).reshape(-1).long()] = \
        torch.arange(B * T, device="cuda")
    token = token[:-1].view(n, 1, ps)
    at = token.clamp(min=0)
    head = torch.arange(H, device="cuda")[None, :, None]
    for pages, rows in ((s["pk"], s["k"]), (s["pv"], s["v"])):
        pages.copy_(torch.where(token[..., None] >= 0, rows[at // T, head, at % T], pages))
    return {"k": s["pk"], "v": s["pv"]}


def _plain_attention(s):
    q, pk, table, lens = s["q"], s["pk"], s["table"], s["lens"]
    B, Hq, D = q.shape
    Hkv, ps = pk.shape[1], pk.shape[2]
    columns = -(-s["longest"] // ps)
    pages = table[:, :columns].clamp(min=0).long()
    k = pk[pages].permute(0, 2, 1, 3, 4).reshape(B, Hkv, columns * ps, D).float()
    seen = torch.arange(columns * ps, device="cuda")[None, None, None, :] < lens[:, None, None, None]
    x = torch.matmul(q.float().view(B, Hkv, Hq // Hkv, D), k.transpose(2, 3)) / math.sqrt(D)
    del k
    x = torch.where(seen, x, torch.full_like(x, NEG))
    m = x.amax(3, keepdim=True)
    p = torch.exp(x - torch.where(m == NEG, torch.zeros_like(m), m))
    v = s["pv"][pages].permute(0, 2, 1, 3, 4).reshape(B, Hkv, columns * ps, D).float()
    v = torch.where(seen.transpose(2, 3), v, torch.zeros_like(v))
    total = p.sum(3, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    return o.reshape(B, Hq, D).to(q.dtype)


def _plain_select(s):
    G, K, n, eos = s["groups"], s["beams"], s["n_out"], s["eos"]
    x = s["logits"].double()
    V = x.shape[1]
    m = x.amax(1, keepdim=True)
    x = x - torch.where(m == NEG, torch.zeros_like(m), m)
    total = torch.exp(x).sum(1, keepdim=True)
    x = x - torch.log(torch.where(total == 0, torch.ones_like(total), total)) + s["scores"].double()[:, None]
    ended = (s["last"] == eos)[:, None]
    end = torch.where(torch.arange(V, device="cuda")[None, :] == eos, s["scores"].double()[:, None],
                      torch.full((1, 1), NEG, device="cuda", dtype=torch.float64))
    x = torch.where(ended, end, x).view(G, K * V)
    # the n largest; among those equal to the smallest of them, the lowest places
    best, at = torch.topk(x, n, dim=1)
    edge = best[:, -1:]
    place = torch.arange(K * V, device="cuda")[None, :]
    tied = torch.topk(torch.where(x == edge, place, torch.full_like(place, K * V)), n, dim=1, largest=False)[0]
    places = torch.cat([torch.where(best > edge, at, torch.full_like(at, K * V)), tied], 1).sort(1)[0]
    values = torch.where(places < K * V, torch.gather(x, 1, places.clamp(max=K * V - 1)),
                         torch.full((1, 1), NEG, device="cuda", dtype=torch.float64))
    order = values.sort(dim=1, descending=True, stable=True)[1][:, :n]
    places, values = torch.gather(places, 1, order), torch.gather(values, 1, order)
    s["parents"].copy_(places // V + K * torch.arange(G, device="cuda")[:, None])
    s["tokens"].copy_(places % V)
    s["best"].copy_(values)
    return {"parents": s["parents"], "tokens": s["tokens"], "scores": s["best"]}


def _plain_reorder(s):
    table, ps, lens = s["table"], s["page"], s["lens"]
    full, rest = lens // ps, lens % ps
    at = full.clamp(max=table.shape[1] - 1).long()[:, None]
    parents = s["parents"].long()
    dst = torch.gather(table, 1, at)[:, 0].long()
    src = dst[parents]
    row = torch.arange(ps, device="cuda")[None, None, None, :, None] < rest[None, :, None, None, None]
    for pages in (s["pk"], s["pv"]):
        pages[:, dst] = torch.where(row, pages[:, src], pages[:, dst])
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    table.copy_(torch.where(col < full[:, None], table[parents], table))
    return {"table": table, "k": s["pk"], "v": s["pv"]}


def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plain_plan, "release": _plain_release, "store": _plain_store, "attention": _plain_attention,
            "select": _plain_select, "reorder": _plain_reorder}[state["op"]](state)


# ----------------------------------------------------------------------------- work and 64-bit results

def work(case):
    op = case["op"]
    es = 2 if case.get("dtype") == "bf16" else 4
    if op in ("plan", "release"):
        B, T, ps = case["batch"], case["tokens"], case["page"]
        counts = _np_spread(case["least"], T, B)
        # ceil((start + count) / page) - ceil(start / page) is count / page on the average over start
        fresh = sum(c / ps if case["held"] else _ceil(c, ps) for c in counts)
        return {"bytes": 8 * B + 8 * fresh + 8 + (4 * B * T if op == "plan" else 0), "flops": 0}
    if op == "store":
        rows = sum(_np_spread(case["least"], case["tokens"], case["batch"]))
        return {"bytes": 4 * rows * case["kv_heads"] * case["dim"] * es + 4 * case["batch"] * case["tokens"],
                "flops": 0}
    if op == "attention":
        keys = sum(_np_spread(case["least"], case["longest"], case["batch"]))
        rows = case["batch"] * case["heads"] * case["dim"]
        return {"bytes": 2 * keys * case["kv_heads"] * case["dim"] * es + 2 * rows * es +
                4 * keys // case["page"] + 4 * case["batch"], "flops": 4 * keys * case["heads"] * case["dim"]}
    if op == "select":
        # a beam at -inf or at its end adds no candidate that its logits decide
        read = case["groups"] * (1 if case["first"] else case["beams"] - case["ended"]) * case["vocab"]
        return {"bytes": 4 * read + 8 * case["groups"] * case["beams"] + 12 * case["groups"] * case["n_out"],
                "flops": 4 * read}
    G, K, ps = case["groups"], case["beams"], case["page"]
    # parents drawn at random: rows whose parent is another row are written, rows that such a row names are read
    written, read = K - 1, K * (1 - (1 - 1 / K) ** (K - 1))
    part = (case["len"] % ps) * case["kv_heads"] * case["dim"] * es * 2 * case["layers"]
    return {"bytes": G * (written + read) * part + G * (written + read) * (case["len"] // ps) * 4 + 8 * G * K,
            "flops": 0}


def exact(case, seed):
    if case["op"] not in ("attention", "select"):
        return None                              # whole numbers and copies: nothing is computed
    s = prepare(case, seed)
    if case["op"] == "attention":
        B, Hq, D = s["q"].shape
        group = Hq // case["kv_heads"]
        out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
        lens = s["lens"].tolist()
        for b in range(B):
            n = lens[b]
            if n == 0:
                continue
            ids = s["table"][b, : _ceil(n, case["page"])].long()
            for g in range(case["kv_heads"]):
                k = s["pk"][ids, g].reshape(-1, D)[:n].double()
                v = s["pv"][ids, g].reshape(-1, D)[:n].double()
                z = (k @ s["q"][b, g * group:(g + 1) * group].double().T) * D ** -0.5
                out[b, g * group:(g + 1) * group] = torch.softmax(z, 0).T @ v
        return out
    G, K, V, n = case["groups"], case["beams"], case["vocab"], case["n_out"]
    parents, tokens, best = np.zeros((G, n), np.int64), np.zeros((G, n), np.int64), np.zeros((G, n))
    scores, last = s["scores"].double().cpu().numpy(), s["last"].cpu().numpy()
    for g in range(G):
        rows = range(g * K, (g + 1) * K)
        c = torch.log_softmax(s["logits"][g * K:(g + 1) * K].double(), 1).cpu().numpy()
        for i, r in enumerate(rows):
            if last[r] == s["eos"]:
                c[i] = -np.inf
                c[i, s["eos"]] = scores[r]
            else:
                c[i] += scores[r]
        c = c.reshape(-1)
        few = np.flatnonzero(c >= np.partition(c, len(c) - n)[len(c) - n])
        pick = few[np.lexsort((few, -c[few]))[:n]]
        parents[g], tokens[g], best[g] = pick // V + g * K, pick % V, c[pick]
    return {"parents": parents, "tokens": tokens, "scores": best}
