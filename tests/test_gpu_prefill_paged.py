"""The block on chunks of new tokens over a paged cache, and a serving round: prompts in chunks, forks, decode steps, log
probabilities, pages given back."""
import numpy as np
import pytest
import torch

import workloads
from oracle import block as ob
from oracle.bf16 import round_bf16
from tests import chunk_ref as ref
from tests.blockrun import BF16_TOL, check_bf16_output

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16


def _ddb():
    import dense_decoder_block_gb300 as ddb
    ddb.lib()
    return ddb


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def block(dims, max_seq, std=0.03):
    ddb = _ddb()
    w, g = workloads.make_weights(dims, weight_std=std)
    dev = torch.device(DEV)
    return ddb, ddb.LlamaBlock(dims, {k: t.to(dev) for k, t in w.items()}, {k: t.to(dev) for k, t in g.items()}, max_seq), w, g


def pages(ddb, dims, batch, max_seq, ps, spare=0):
    columns = max_seq // ps
    n = batch * columns + spare
    k, v = (torch.full((n, dims.n_kv_heads, ps, 128), float("nan"), dtype=BF, device=DEV) for _ in range(2))
    table = torch.randperm(n, generator=torch.Generator().manual_seed(2))[:batch * columns].view(batch, columns)
    return ddb.PagedCache(k, v), table.to(torch.int32).contiguous().to(DEV)


def rows_of(pages_, table, b, n, ps):
    ids = table[b, :ref.ceil_div(n, ps)].long()
    return pages_[ids].transpose(0, 1).reshape(pages_.shape[1], -1, 128)[:, :n]


SMALL = workloads.BlockDims(512, 8, 2, 128, 1024)
WIDE = workloads.BlockDims(d_model=2048, n_heads=16, n_kv_heads=1, head_dim=128, d_ff=1024)
GROUP3 = workloads.BlockDims(768, 6, 2, 128, 512)


# chunks of two calls: start and count of each sequence; rows 3 x 7 (weight-streaming), 3 x 50, 2 x 400 (token-tiled)
@pytest.mark.parametrize("dims", [SMALL, WIDE, GROUP3], ids=["group4", "group16", "group3"])
@pytest.mark.parametrize("counts", [([5, 0, 7], [3, 7, 1]), ([50, 17, 33], [1, 50, 20]), ([400, 129], [300, 128])],
                         ids=["few", "some", "many"])
@pytest.mark.parametrize("ps", [16, 128])
def test_chunks_agree_with_the_contiguous_prefill(dims, counts, ps):
    """Two calls of ragged chunks: cache rows bit for bit those of prefill_at, outputs within the block's parity bound."""
    max_seq = 1024
    ddb, blk, _, _ = block(dims, max_seq)
    B = len(counts[0])
    kv, table = pages(ddb, dims, B, max_seq, ps)
    before = (kv.k.clone(), kv.v.clone())
    start, total = [0] * B, [a + b for a, b in zip(*counts)]
    T0 = max(total)
    x = workloads.make_x(B, T0, dims.d_model).to(DEV)
    got = [[] for _ in range(B)]
    for count in counts:
        T = max(count)
        xc = torch.full((B, T, dims.d_model), float("nan"), dtype=BF, device=DEV)     # padding holds anything
        for b in range(B):
            xc[b, :count[b]] = x[b, start[b]:start[b] + count[b]]
        y = torch.empty_like(xc)
        blk.prefill_paged(xc, kv, table, _i32(start), _i32(count), y, blk.workspace_paged(B, T))
        assert blk.poll_error() == 0
        for b in range(B):
            got[b].append(y[b, :count[b]])
        start = [s + c for s, c in zip(start, count)]
    for b in range(B):
        n = total[b]
        kc = torch.zeros(1, dims.n_kv_heads, max_seq, 128, dtype=BF, device=DEV)
        cache = ddb.KVCache(kc, torch.zeros_like(kc))
        want = torch.empty(1, n, dims.d_model, dtype=BF, device=DEV)
        blk.prefill(x[b:b + 1, :n].contiguous(), cache, want, blk.workspace(1, n))
        assert torch.equal(rows_of(kv.k, table, b, n, ps), cache.k[0, :, :n])
        assert torch.equal(rows_of(kv.v, table, b, n, ps), cache.v[0, :, :n])
        # the bound is that of one result to the exact one, e: |a - b| <= |a - e| + |b - e|, twice it between two results
        check_bf16_output(workloads.to_numpy64(torch.cat(got[b])), workloads.to_numpy64(want[0]), 2 * BF16_TOL,
                          what=f"chunks of sequence {b}")
    # no other row was written
    for a, z, name in ((kv.k, before[0], "k"), (kv.v, before[1], "v")):
        written = ~torch.isnan(a.float()).all(-1)[:, 0]
        assert int(written.sum()) == sum(total), name


@pytest.mark.parametrize("dims", [SMALL, WIDE, GROUP3], ids=["group4", "group16", "group3"])
def test_against_the_oracle(dims):
    max_seq, ps = 256, 16
    ddb, blk, w, g = block(dims, max_seq)
    kv, table = pages(ddb, dims, 1, max_seq, ps)
    T = 150
    x = workloads.make_x(1, T, dims.d_model)
    ys = []
    for s, c in ((0, 100), (100, 50)):
        xc = x[:, s:s + c].contiguous().to(DEV)
        y = torch.empty_like(xc)
        blk.prefill_paged(xc, kv, table, _i32([s]), _i32([c]), y, blk.workspace_paged(1, c))
        ys.append(y)
    assert blk.poll_error() == 0
    to64 = workloads.to_numpy64
    kc = np.zeros((1, dims.n_kv_heads, max_seq, 128))
    want = ob.block_forward(to64(x), {k: to64(t) for k, t in w.items()}, {k: to64(t) for k, t in g.items()}, dims, kc,
                            np.zeros_like(kc), 0, round_bf16)
    check_bf16_output(to64(torch.cat(ys, 1)), want, what="paged prefill against the oracle")


def test_records_bad_words_and_pages():
    ddb, blk, _, _ = block(SMALL, 64)
    kv, table = pages(ddb, SMALL, 2, 64, 16)
    x = workloads.make_x(2, 8, 512).to(DEV)
    y, ws = torch.empty_like(x), blk.workspace_paged(2, 8)

    def run(start, count, t=table):
        kv.k.fill_(0)
        kv.v.fill_(0)
        blk.prefill_paged(x, kv, t, _i32(start), _i32(count), y, ws)
        rc = blk.poll_error()
        return rc, rows_of(kv.k, table, 0, 64, 16).abs().sum((0, 2)), y.clone()
    rc, rows, good = run([3, 30], [8, 5])
    assert rc == 0 and bool((rows[3:11] > 0).all()) and not rows[11:].any() and not rows[:3].any()
    for s, c in ((57, 8), (-1, 8), (3, 9), (3, -1), (2 ** 31 - 1, 8)):
        rc, rows, y1 = run([s, 30], [c, 5])
        assert rc == -3 and not rows.any() and torch.equal(y1[1, :5], good[1, :5])
    bad = table.clone()
    bad[0, 0] = kv.n_pages
    rc, rows, y1 = run([12, 30], [8, 5], bad)         # positions 12 .. 15 on the bad page, 16 .. 19 on the next
    assert rc == -1 and not rows[:16].any() and bool((rows[16:20] > 0).all()) and torch.equal(y1[1, :5], good[1, :5])
    with pytest.raises(ddb.LlamaError):
        blk.prefill_paged(x, kv, table, _i32([0, 0]), _i32([1, 1]), y, ws[:-1024])
    ddb.llama_block_prefill_paged(blk.h, x, 0, 8, kv.c, table, _i32([0]), _i32([0]), y, ws, ws.numel())


def test_replayed_as_a_graph():
    """A captured chunk call whose starts and counts move between replays."""
    ddb, blk, _, _ = block(SMALL, 512)
    kv, table = pages(ddb, SMALL, 2, 512, 16)
    T = 40
    x = workloads.make_x(2, 4 * T, 512).to(DEV)
    xs, y = x[:, :T].clone(), torch.empty(2, T, 512, dtype=BF, device=DEV)
    start, count, ws = _i32([0, 0]), _i32([T, T]), blk.workspace_paged(2, T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        blk.prefill_paged(xs, kv, table, start, count, y, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        blk.prefill_paged(xs, kv, table, start, count, y, ws)
    kv2, _ = pages(ddb, SMALL, 2, 512, 16)
    for i in range(4):
        xs.copy_(x[:, i * T:(i + 1) * T])
        start.fill_(i * T)
        graph.replay()
        y2 = torch.empty_like(y)
        blk.prefill_paged(xs, kv2, table, start, count, y2, blk.workspace_paged(2, T))
        torch.cuda.synchronize()
        assert torch.equal(y, y2)
    assert blk.poll_error() == 0 and torch.equal(rows_of(kv.k, table, 1, 4 * T, 16), rows_of(kv2.k, table, 1, 4 * T, 16))


def test_a_serving_round():
    """Two prompts in ragged chunks on pages (plan, paged prefill), three samples of the first and one of the second (fork),
    decode steps on all of them, the log probabilities of their tokens, and the end of all rows: what a sample sees is what
    a row that was prefilled by itself sees, bit for bit, and the pool ends as it began."""
    dims, max_seq, ps, rows, vocab = SMALL, 256, 16, 8, 1024
    ddb, blk, _, _ = block(dims, max_seq)
    n_pages, columns = 100, max_seq // ps
    k = torch.zeros(n_pages, dims.n_kv_heads, ps, 128, dtype=BF, device=DEV)
    kv = ddb.PagedCache(k, torch.zeros_like(k))
    caches = ddb.PagedCacheList([kv])
    free, pool = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(DEV), _i32([n_pages, 0])
    free0 = free.clone()
    refs, err = torch.zeros(n_pages, dtype=torch.int32, device=DEV), _i32([0])
    table = torch.full((rows, columns), -1, dtype=torch.int32, device=DEV)
    w_out = (torch.randn(vocab, dims.d_model, generator=torch.Generator().manual_seed(3)) * 0.05).to(BF).to(DEV)
    gain = torch.ones(dims.d_model, dtype=BF, device=DEV)
    x = workloads.make_x(2, 120, dims.d_model).to(DEV)
    start = [0, 0]
    for count in ([60, 17], [40, 37]):
        st, ct = _i32(start), _i32(count)
        slots = torch.empty(2, max(count), dtype=torch.int32, device=DEV)
        ddb.llama_paged_plan(st, ct, ps, n_pages, free, pool, table[:2], slots, err_dev=err)
        xc = torch.zeros(2, max(count), dims.d_model, dtype=BF, device=DEV)
        for b in range(2):
            xc[b, :count[b]] = x[b, start[b]:start[b] + count[b]]
        blk.prefill_paged(xc, kv, table[:2], st, ct, torch.empty_like(xc), blk.workspace_paged(2, max(count)))
        start = [a + b for a, b in zip(start, count)]
    assert start == [100, 54]
    # samples: rows 2, 3, 4 of prompt 0, row 6 of prompt 1
    src, dst, lens = _i32([0, 0, 0, 1]), _i32([2, 3, 4, 6]), _i32([100, 100, 100, 54])
    ws = torch.empty(max(ddb.llama_paged_fork_workspace_bytes(4), ddb.llama_paged_free_workspace_bytes(8, n_pages)),
                     dtype=torch.uint8, device=DEV)
    ddb.llama_paged_fork(src, dst, lens, refs, free, pool, table, caches, ws, err_dev=err)
    live = [0, 1, 2, 3, 4, 6]
    lens = [100, 54, 100, 100, 100, 54]
    tables = table[live].contiguous()
    # a decode step for each: the same token for rows of one prompt gives the same bits; the new rows lie in pages of their own
    xd = torch.stack([x[0, 110], x[1, 110], x[0, 110], x[0, 110], x[0, 111], x[1, 110]])[:, None].contiguous()
    yd = torch.empty_like(xd)
    steps = _i32(lens)
    slots = torch.empty(6, 1, dtype=torch.int32, device=DEV)
    ddb.llama_paged_plan(steps, torch.ones_like(steps), ps, n_pages, free, pool, tables, slots, err_dev=err)
    assert len(set(slots.flatten().tolist())) == 6
    blk.decode_paged(xd, kv, tables, steps, yd, blk.workspace(6, 1))
    assert blk.poll_error() == 0 and int(err) == 0
    assert torch.equal(yd[0], yd[2]) and torch.equal(yd[0], yd[3]) and torch.equal(yd[1], yd[5]) and not torch.equal(yd[0], yd[4])
    # and so does the same token as a chunk of one
    yc = torch.empty_like(xd)
    blk.prefill_paged(xd, kv, tables, steps, torch.ones_like(steps), yc, blk.workspace_paged(6, 1))
    check_bf16_output(workloads.to_numpy64(yc), workloads.to_numpy64(yd), 2 * BF16_TOL, what="one token as a chunk")
    assert torch.equal(yc[0], yc[2])
    # log probabilities of the chosen tokens
    ids = torch.empty(6, dtype=torch.int32, device=DEV)
    logits = torch.empty(6, vocab, device=DEV)
    head = torch.empty(ddb.llama_lmhead_workspace_bytes(6, dims.d_model, vocab), dtype=torch.uint8, device=DEV)
    ddb.llama_lmhead_argmax(yd, 6, dims.d_model, gain, w_out, vocab, dims.d_model, 1e-5, ids, logits, head, head.numel())
    lp, top, best = torch.empty(6, device=DEV), torch.empty(6, 3, dtype=torch.int32, device=DEV), torch.empty(6, 3, device=DEV)
    ddb.llama_token_logprobs(logits, ids, lp, top_ids=top, top_logprobs=best)
    assert torch.equal(top[:, 0], ids) and torch.equal(best[:, 0], lp)
    want = torch.log_softmax(logits.double(), 1).gather(1, ids.long()[:, None])[:, 0]
    assert float((lp.double() - want).abs().max()) <= ref.logprob_tol(10.0, np.array([0.0, 20.0]), vocab).max()
    # the end: samples first, then the prompts
    table[live] = tables
    held = _i32([n + 1 for n in lens])
    for part in ([2, 4, 5], [0, 1, 3]):
        r = _i32([live[i] for i in part])
        ddb.llama_paged_free(r, held[part].contiguous(), ps, n_pages, refs, free, pool, table, ws, err_dev=err)
    assert pool.tolist() == [n_pages, 0] and int(err) == 0 and not refs.any()
    assert sorted(free.tolist()) == sorted(free0.tolist())
