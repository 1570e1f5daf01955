"""Cases of the operators that serve prompts in chunks on shared pages: inputs, plain forms, the library's calls and
64-bit results.

Four calls that a serving loop runs together: llama_paged_chunk_attention (a chunk of new tokens per sequence over the
paged cache), llama_token_logprobs (log probabilities of given tokens with entropy and top alternatives), and
llama_paged_fork with llama_paged_free (samples of a prompt share its pages, and give them up).

Sizes: the 8B block (32 / 8 heads of 128, vocabulary 128,256, 32 layers, batch 32 near 1000 cached positions), the 70B
block (64 / 8 heads, prefill of 4096 tokens, 8192 positions) and the tiny fp32 block (4 / 2 heads of 64, 16 tokens) of
this repository, and generic page sizes, batches and lengths.
"""
import math

import torch

own = False

VOCAB = 128256
NEG = float("-inf")


def listed():
    return [
        # the tiny fp32 block's prefill of 16 tokens, two prompts: the smallest call, latency alone
        {"name": "chunk_tiny_f32", "op": "chunk", "batch": 2, "tokens": 16, "heads": 4, "kv_heads": 2, "dim": 64,
         "dtype": "f32", "page": 16, "held": 4, "held_least": 0, "least": 16},
        # four drafted tokens of each of 32 requests near 1000 cached positions are verified at once (8B heads)
        {"name": "chunk_verify", "op": "chunk", "batch": 32, "tokens": 4, "heads": 32, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "page": 16, "held": 1056, "held_least": 944, "least": 1},
        # the next turn of one long conversation (8B heads): few rows, a long cache
        {"name": "chunk_turn", "op": "chunk", "batch": 1, "tokens": 100, "heads": 32, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "page": 64, "held": 8192, "held_least": 8192, "least": 100},
        # one scheduler step: chunks of up to 512 tokens of 8 prompts, some just begun, some far along (8B heads)
        {"name": "chunk_ragged", "op": "chunk", "batch": 8, "tokens": 512, "heads": 32, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "page": 16, "held": 2048, "held_least": 0, "least": 37},
        # the second half of a prompt of 8192 tokens (70B heads)
        {"name": "chunk_70b", "op": "chunk", "batch": 1, "tokens": 4096, "heads": 64, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "page": 128, "held": 4096, "held_least": 4096, "least": 4096},
        # one answer's token with the 20 best alternatives
        {"name": "logprobs_one", "op": "logprobs", "rows": 1, "vocab": VOCAB, "top": 20, "masked": 0.0, "skipped": 0},
        # one decode step of the benchmark's batch, 5 alternatives each, constrained answers: half the tokens masked
        {"name": "logprobs_step", "op": "logprobs", "rows": 32, "vocab": VOCAB, "top": 5, "masked": 0.5, "skipped": 0},
        # scoring: a padded chunk of 1024 rows of given tokens, some of them padding
        {"name": "logprobs_prompt", "op": "logprobs", "rows": 1024, "vocab": VOCAB, "top": 1, "masked": 0.0,
         "skipped": 100},
        # one prompt sampled four times: three forks on all 32 layers of the 8B stack, freed again
        {"name": "fork_one", "op": "fork", "prompts": 1, "forks": 3, "layers": 32, "page": 16, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "len": 1000, "len_least": 1000},
        # 16 prompts sampled eight times each, 32 layers
        {"name": "fork_batch", "op": "fork", "prompts": 16, "forks": 7, "layers": 32, "page": 16, "kv_heads": 8,
         "dim": 128, "dtype": "bf16", "len": 1031, "len_least": 250},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "logprobs", "logprobs", "fork"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "chunk":
        bf16 = rng.random() < 0.8
        kv_heads = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 8, 16] if bf16 else [1, 2, 3, 4])
        heads = kv_heads * group
        held, tokens, batch = _log(rng, 1, 65536), _log(rng, 1, 4096), _log(rng, 1, 64)
        most = (1 << 30) if bf16 else (1 << 25)       # scores of a padded batch
        tokens = max(1, min(tokens, most // (heads * (held + tokens))))
        held = min(held, most // (heads * tokens))
        batch = max(1, min(batch, most // (heads * tokens * (held + tokens)), (1 << 19) // (kv_heads * (held + tokens))))
        return {"op": op, "batch": batch, "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
                "dim": 128 if bf16 else rng.choice([32, 64, 128]), "dtype": "bf16" if bf16 else "f32", "page": page,
                "held": held, "held_least": rng.choice([0, held // 2, held]), "least": rng.choice([0, 1, tokens])}
    if op == "logprobs":
        rows, vocab = _log(rng, 1, 1024), _log(rng, 100, VOCAB)
        return {"op": op, "rows": rows, "vocab": vocab, "top": rng.choice([0, 1, 5, 20, rng.randint(1, 32)]),
                "masked": rng.choice([0.0, 0.0, 0.5]), "skipped": rng.choice([0, 0, rows // 3])}
    length = _log(rng, 1, 2000)
    return {"op": op, "prompts": _log(rng, 1, 16), "forks": rng.randint(1, 7), "layers": _log(rng, 1, 32), "page": page,
            "kv_heads": rng.choice([1, 2, 4, 8]), "dim": 128, "dtype": "bf16", "len": length,
            "len_least": rng.choice([1, max(1, length // 2), length])}


# ----------------------------------------------------------------------------- inputs

def _np_spread(least, most, n):
    return [least + i * (most - least) // (n - 1) for i in range(n)] if n > 1 else [most]


def _spread(least, most, n, gen):
    """n whole numbers spread evenly over least .. most, in an order from the seed."""
    v = torch.tensor(_np_spread(least, most, n), device="cuda")
    return v[torch.randperm(n, generator=gen, device="cuda")].to(torch.int32)


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


def _prepare_chunk(case, gen):
    B, T, ps = case["batch"], case["tokens"], case["page"]
    start = _spread(case["held_least"], case["held"], B, gen)
    count = _spread(case["least"], T, B, gen)
    need = (start + count + ps - 1) // ps
    longest = case["held"] + T
    n_pages = max(1, int(need.sum()) + 3)
    shape = (n_pages, case["kv_heads"], ps, case["dim"])
    pk, pv = (torch.randn(shape, generator=gen, device="cuda", dtype=_dtype(case)) for _ in range(2))
    q = torch.randn(B, T, case["heads"], case["dim"], generator=gen, device="cuda", dtype=_dtype(case))
    return {"q": q, "pk": pk, "pv": pv, "table": _tables(need, _ceil(longest, ps) + 1, n_pages, gen), "start": start,
            "count": count, "longest": longest, "o": torch.zeros_like(q)}


def _prepare_logprobs(case, gen):
    R, V, n = case["rows"], case["vocab"], case["top"]
    logits = torch.randn(R, V, generator=gen, device="cuda") * 3.0
    if case["masked"]:
        logits[torch.rand(R, V, generator=gen, device="cuda") < case["masked"]] = NEG
    # the given tokens: drawn from the distribution of each row
    tokens = torch.empty(R, dtype=torch.int32, device="cuda")
    for r in range(0, R, 256):
        part = logits[r:r + 256]
        noise = -torch.log(-torch.log(torch.rand(part.shape, generator=gen, device="cuda").clamp(1e-20, 1 - 1e-7)))
        tokens[r:r + 256] = (part + noise).argmax(1).to(torch.int32)
    off = torch.randperm(R, generator=gen, device="cuda")[:case["skipped"]]
    tokens[off] = -1
    return {"logits": logits, "tokens": tokens, "n": n, "logprobs": torch.zeros(R, device="cuda"),
            "entropy": torch.zeros(R, device="cuda"),
            "top_ids": torch.zeros(R, n, dtype=torch.int32, device="cuda"),
            "top_logprobs": torch.zeros(R, n, device="cuda")}


def _prepare_fork(case, gen):
    P, F, ps = case["prompts"], case["forks"], case["page"]
    lens = _spread(case["len_least"], case["len"], P, gen)
    need = (lens + ps - 1) // ps
    columns = _ceil(case["len"], ps) + 2
    used = int(need.sum())
    n_pages = used + P * F + 5
    # rows 0 .. P-1 hold the prompts, the rows of their forks follow in an order from the seed
    table = _tables(torch.cat([need, torch.zeros(P * F, dtype=need.dtype, device="cuda")]), columns, n_pages, gen)
    taken = torch.zeros(n_pages, dtype=torch.bool, device="cuda")
    taken[table[table >= 0].long()] = True
    order = torch.randperm(n_pages, generator=gen, device="cuda")
    free = order[~taken[order]].to(torch.int32)
    pool = torch.tensor([free.numel(), 0], dtype=torch.int32, device="cuda")
    free = torch.cat([free, torch.full((used,), -1, dtype=torch.int32, device="cuda")]).contiguous()
    src = torch.arange(P * F, device="cuda", dtype=torch.int32) // F
    # every third prompt is shared with one more row already (another call's sample)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    shared = table[:P][::3]
    refs[shared[shared >= 0].long()] = 1
    shape = (case["layers"], n_pages, case["kv_heads"], ps, case["dim"])
    pk, pv = (torch.randn(shape, generator=gen, device="cuda", dtype=_dtype(case)) for _ in range(2))
    return {"src": src, "dst": (P + torch.randperm(P * F, generator=gen, device="cuda")).to(torch.int32),
            "lens": lens[src.long()].contiguous(), "table": table, "free": free, "pool": pool, "refs": refs,
            "pool_mid": torch.zeros(2, dtype=torch.int32, device="cuda"),
            "pool_out": torch.zeros(2, dtype=torch.int32, device="cuda"), "pk": pk, "pv": pv, "n_pages": n_pages}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    state = {"chunk": _prepare_chunk, "logprobs": _prepare_logprobs, "fork": _prepare_fork}[op](case, gen)
    state["op"], state["page"] = op, case.get("page", 0)
    state["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:
        import dense_decoder_block_gb300 as ddb
        state["ddb"] = ddb
        need = 0
        if op == "chunk":
            state["cache"] = ddb.PagedCache(state["pk"], state["pv"])
            need = ddb.llama_paged_chunk_attention_workspace_bytes(case["batch"], case["tokens"], case["heads"],
                                                                   case["kv_heads"], case["dim"], state["longest"])
        if op == "fork":
            state["cache"] = ddb.PagedCacheList([ddb.PagedCache(k, v) for k, v in zip(state["pk"], state["pv"])])
            need = max(ddb.llama_paged_fork_workspace_bytes(state["src"].numel()),
                       ddb.llama_paged_free_workspace_bytes(state["src"].numel(), state["n_pages"]))
        state["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return state


# ----------------------------------------------------------------------------- the library's calls

def _run_own(s):
    ddb, op = s["ddb"], s["op"]
    if op == "chunk":
        ddb.llama_paged_chunk_attention(s["q"], s["cache"], s["table"], s["start"], s["count"], s["longest"], s["o"],
                                        s["ws"], err_dev=s["err"])
        return s["o"]
    if op == "logprobs":
        ddb.llama_token_logprobs(s["logits"], s["tokens"], s["logprobs"], entropy=s["entropy"],
                                 top_ids=s["top_ids"] if s["n"] else None,
                                 top_logprobs=s["top_logprobs"] if s["n"] else None, err_dev=s["err"])
        return {"logprobs": s["logprobs"], "entropy": s["entropy"], "ids": s["top_ids"], "top": s["top_logprobs"]}
    # the forks of a round of sampling, and their end
    ddb.llama_paged_fork(s["src"], s["dst"], s["lens"], s["refs"], s["free"], s["pool"], s["table"], s["cache"], s["ws"],
                         pool_out=s["pool_mid"], err_dev=s["err"])
    ddb.llama_paged_free(s["dst"], s["lens"], s["page"], s["n_pages"], s["refs"], s["free"], s["pool_mid"], s["table"],
                         s["ws"], pool_out=s["pool_out"], err_dev=s["err"])
    return _fork_result(s)


def _fork_result(s):
    return {"table": s["table"], "refs": s["refs"], "pages": s["free"], "forked": s["pool_mid"][:1],
            "freed": s["pool_out"][:1], "k": s["pk"], "v": s["pv"]}


# ----------------------------------------------------------------------------- plain forms

def _plain_chunk(s):
    q, table = s["q"], s["table"]
    B, T, Hq, D = q.shape
    Hkv, ps = s["pk"].shape[1], s["pk"].shape[2]
    columns = -(-s["longest"] // ps)
    L = columns * ps
    pages = table[:, :columns].clamp(min=0).long()
    k = s["pk"][pages].permute(0, 2, 1, 3, 4).reshape(B, Hkv, 1, L, D).float()
    qf = q.float().view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    x = torch.matmul(qf, k.transpose(3, 4)) / math.sqrt(D)                       # [B, Hkv, group, T, L]
    del k
    t = torch.arange(T, device="cuda")
    last = (s["start"][:, None] + t[None, :])[:, None, None, :, None]
    x.masked_fill_(torch.arange(L, device="cuda") > last, NEG)                   # key 0 is seen by every token
    p = torch.exp(x.sub_(x.amax(4, keepdim=True)))
    del x
    end = (s["start"] + s["count"])[:, None, None, None, None]
    v = s["pv"][pages].permute(0, 2, 1, 3, 4).reshape(B, Hkv, 1, L, D).float()
    v = torch.where(torch.arange(L, device="cuda")[:, None] < end, v, torch.zeros_like(v))
    o = torch.matmul(p, v) / p.sum(4, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D).to(q.dtype)
    s["o"].copy_(torch.where((t[None, :] < s["count"][:, None])[:, :, None, None], o, s["o"]))
    return s["o"]


def _plain_logprobs(s):
    x, n = s["logits"], s["n"]
    on = s["tokens"] >= 0
    m = x.amax(1, keepdim=True)
    e = torch.exp((x - m).double())
    total = e.sum(1)
    lse = torch.log(total)
    at = s["tokens"].clamp(min=0).long()[:, None]
    logprobs = (torch.gather(x, 1, at) - m)[:, 0].double() - lse
    weighted = torch.where(e > 0, e * (x - m).double(), torch.zeros_like(e)).sum(1)
    entropy = lse - weighted / total
    s["logprobs"].copy_(torch.where(on, logprobs.float(), s["logprobs"]))
    s["entropy"].copy_(torch.where(on, entropy.float(), s["entropy"]))
    if n:
        # the n largest; among those equal to the smallest of them, the lowest places
        V = x.shape[1]
        best, place = torch.topk(x, n, dim=1)
        edge = best[:, -1:]
        col = torch.arange(V, device="cuda")[None, :]
        tied = torch.topk(torch.where(x == edge, col, torch.full_like(col, V)), n, dim=1, largest=False)[0]
        places = torch.cat([torch.where(best > edge, place, torch.full_like(place, V)), tied], 1).sort(1)[0]
        values = torch.where(places < V, torch.gather(x, 1, places.clamp(max=V - 1)), torch.full_like(edge, NEG))
        values = torch.where(places < V, values, torch.full_like(values, float("-inf")))
        order = values.sort(dim=1, descending=True, stable=True)[1][:, :n]
        places, values = torch.gather(places, 1, order), torch.gather(values, 1, order)
        top = (values - m).double() - lse[:, None]
        s["top_ids"].copy_(torch.where(on[:, None], places.int(), s["top_ids"]))
        s["top_logprobs"].copy_(torch.where(on[:, None], top.float(), s["top_logprobs"]))
    return {"logprobs": s["logprobs"], "entropy": s["entropy"], "ids": s["top_ids"], "top": s["top_logprobs"]}


def _plain_fork(s):
    ps, table, refs, free = s["page"], s["table"], s["refs"], s["free"]
    src, dst, lens = s["src"].long(), s["dst"].long(), s["lens"]
    columns = table.shape[1]
    col = torch.arange(columns, device="cuda")[None, :]
    full, rest = (lens // ps)[:, None], lens % ps
    # fork: a page from the stack for every unfilled one, in the order of the forks
    fresh = (rest > 0).int()
    off = torch.cumsum(fresh, 0) - fresh
    page = free[(s["pool"][0] - 1 - off).clamp(min=0).long()]
    old = table[src]
    shares = col < full
    refs.scatter_add_(0, old.clamp(min=0).reshape(-1).long(), shares.reshape(-1).int())
    table[dst] = torch.where(shares, old, torch.where((col == full) & (rest[:, None] > 0), page[:, None], table[dst]))
    at = torch.gather(old, 1, full.clamp(max=columns - 1).long())[:, 0].clamp(min=0).long()
    to = torch.where(rest > 0, page, at).long()              # without an unfilled page: onto itself, no row of it
    row = torch.arange(ps, device="cuda")[None, None, None, :, None] < rest[None, :, None, None, None]
    for pages in (s["pk"], s["pv"]):
        pages[:, to] = torch.where(row, pages[:, at], pages[:, to])
    s["pool_mid"][0] = s["pool"][0] - fresh.sum()
    # free: a row gives up its hold on each of its pages; a page without a holder goes back at its last listing
    entries = table[dst]
    held = (col < ((lens + ps - 1) // ps)[:, None]).reshape(-1)
    entries = entries.clamp(min=0).reshape(-1).long()
    place = torch.arange(entries.numel(), device="cuda")
    drops = torch.zeros_like(refs).scatter_add_(0, entries, held.int())
    last = torch.full((s["n_pages"],), -1, device="cuda").scatter_reduce_(
        0, entries, torch.where(held, place, torch.full_like(place, -1)), "amax")
    back = held & (last[entries] == place) & (drops[entries] > refs[entries])
    number = torch.cumsum(back, 0) - 1
    spot = s["pool_mid"][0] + back.sum() - 1 - number
    spare = torch.cat([free, free[:1]])                      # the place behind the stack takes what does not go back
    spare[torch.where(back, spot, torch.full_like(spot, free.numel())).long()] = entries.int()
    free.copy_(spare[:-1])
    refs.copy_((refs - drops).clamp(min=0))
    s["pool_out"][0] = s["pool_mid"][0] + back.sum()
    return _fork_result(s)


def run(state):
    if own:
        return _run_own(state)
    return {"chunk": _plain_chunk, "logprobs": _plain_logprobs, "fork": _plain_fork}[state["op"]](state)


# ----------------------------------------------------------------------------- work and 64-bit results

def work(case):
    es = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "chunk":
        B, T, D = case["batch"], case["tokens"], case["dim"]
        # starts and counts are spread in orders of their own: their products are taken at the means
        starts, counts = _np_spread(case["held_least"], case["held"], B), _np_spread(case["least"], T, B)
        start = sum(starts) / B
        keys = sum(start + c for c in counts if c > 0)
        rows = sum(counts)
        seen = sum(c * start + c * (c + 1) / 2 for c in counts)
        return {"bytes": 2 * keys * case["kv_heads"] * D * es + 2 * rows * case["heads"] * D * es +
                4 * keys / case["page"] + 8 * B, "flops": 4 * seen * case["heads"] * D}
    if case["op"] == "logprobs":
        rows = case["rows"] - case["skipped"]
        return {"bytes": 4 * rows * case["vocab"] + 4 * case["rows"] + rows * (8 + 8 * case["top"]),
                "flops": 6 * rows * case["vocab"]}
    P, F, ps = case["prompts"], case["forks"], case["page"]
    lens = _np_spread(case["len_least"], case["len"], P)
    row = case["kv_heads"] * case["dim"] * es * 2 * case["layers"]
    moved = sum((n % ps) * row * (1 + F) for n in lens)               # read once, written for every fork
    entries = sum((n // ps) * (4 + F * 8) + F * 12 * (n % ps > 0) for n in lens)
    counts = sum((n // ps) * 16 for n in lens)                         # read and written by both calls
    return {"bytes": moved + entries + counts + 24 * P * F, "flops": 0}


def exact(case, seed):
    if case["op"] == "fork":
        return None                                    # whole numbers and copies: nothing is computed
    s = prepare(case, seed)
    if case["op"] == "chunk":
        B, T, Hq, D = s["q"].shape
        group = Hq // case["kv_heads"]
        out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
        for b, (first, n) in enumerate(zip(s["start"].tolist(), s["count"].tolist())):
            if n == 0:
                continue
            ids = s["table"][b, :_ceil(first + n, case["page"])].long()
            hidden = torch.arange(first + n, device="cuda")[None, :] > first + torch.arange(n, device="cuda")[:, None]
            for g in range(case["kv_heads"]):
                k = s["pk"][ids, g].reshape(-1, D)[:first + n].double()
                v = s["pv"][ids, g].reshape(-1, D)[:first + n].double()
                for h in range(g * group, (g + 1) * group):
                    z = (s["q"][b, :n, h].double() @ k.T) * D ** -0.5
                    out[b, :n, h] = torch.softmax(z.masked_fill_(hidden, NEG), 1) @ v
        return out
    R, n = case["rows"], case["top"]
    out = {"logprobs": torch.zeros(R, dtype=torch.float64, device="cuda"),
           "entropy": torch.zeros(R, dtype=torch.float64, device="cuda"),
           "ids": torch.zeros(R, n, dtype=torch.int64, device="cuda"),
           "top": torch.zeros(R, n, dtype=torch.float64, device="cuda")}
    for r, token in enumerate(s["tokens"].tolist()):
        if token < 0:
            continue
        lp = torch.log_softmax(s["logits"][r].double(), 0)
        out["logprobs"][r] = lp[token]
        out["entropy"][r] = -torch.special.xlogy(lp.exp(), lp.exp()).sum()
        if n:
            value, place = torch.sort(s["logits"][r], descending=True, stable=True)
            out["ids"][r] = place[:n]
            out["top"][r] = lp[place[:n]]
    return out
