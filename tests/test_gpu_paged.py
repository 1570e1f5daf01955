"""The paged KV cache on the GPU: plan, release, store and the attention of one new
token, against plain references (tests/paged_ref.py), and the paged decode step of a
block against its contiguous one, bit for bit."""
import numpy as np
import pytest
import torch

import workloads
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _ddb():
    import dense_decoder_block_gb300 as ddb
    ddb.lib()
    return ddb


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


# ----------------------------------------------------------------------------- plan and release

def _plan_state(start, count, tokens, ps, columns, spare, seed):
    """Random page order; the pages that `start` holds are in the table, -1 behind them."""
    rng = np.random.default_rng(seed)
    n_pages = max(1, len(start) * columns + spare)
    order = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(start), columns), -1, np.int32)
    used = 0
    for b, s in enumerate(start):
        held = min(columns, ref.ceil_div(max(s, 0), ps))
        table[b, :held] = order[used:used + held]
        used += held
    free = np.full(n_pages, -7, np.int32)
    free[:n_pages - used] = order[used:]
    return n_pages, table, free, n_pages - used


def _run_plan(ddb, start, count, tokens, ps, n_pages, table, free, n_free, out=False, release=False):
    t, f, p = _i32(table), _i32(free), _i32([n_free, 0])
    q = _i32([-5, 0]) if out else None
    err = _i32([0])
    slots = torch.full((len(start), tokens), -9, dtype=torch.int32, device=DEV)
    if release:
        ddb.llama_paged_release(_i32(start), _i32(count), ps, n_pages, f, p, t, pool_out=q, err_dev=err)
    else:
        ddb.llama_paged_plan(_i32(start), _i32(count), ps, n_pages, f, p, t, slots, pool_out=q, err_dev=err)
    torch.cuda.synchronize()
    got = (q if out else p).tolist()
    assert got[1] == 0
    if out:
        assert p.tolist() == [n_free, 0]
    return t.cpu().numpy(), slots.cpu().numpy(), f.cpu().numpy(), got[0], int(err[0])


def _same(got, want):
    for x, y in zip(got[:3], want[:3]):
        assert np.array_equal(x, y)
    assert got[3] == want[3] and got[4] == want[4]


PLANS = {
    "one-token": ([0], [1], 1, 16),
    "nothing": ([5], [0], 1, 16),
    "step": (list(range(0, 70)), [1] * 70, 1, 16),
    "ragged": ([0, 0, 33, 16, 15, 0, 700], [17, 0, 31, 16, 1, 32, 45], 45, 16),
    "wide": ([0, 3, 128], [5000, 4097, 1], 5000, 128),
    "many": ([(7 * i) % 300 for i in range(2500)], [(13 * i) % 5 for i in range(2500)], 4, 32),
    "big-pages": ([0, 1023, 1024], [1024, 2, 1], 1024, 1024),
}


@pytest.mark.parametrize("name", PLANS)
@pytest.mark.parametrize("out", [False, True], ids=["in-place", "pool-out"])
def test_plan_then_release(name, out):
    ddb = _ddb()
    start, count, tokens, ps = PLANS[name]
    columns = max(ref.ceil_div(s + c, ps) for s, c in zip(start, count)) + 1
    n_pages, table, free, n_free = _plan_state(start, count, tokens, ps, columns, 3, 1)
    want = ref.plan(start, count, tokens, ps, n_pages, free, n_free, table)
    got = _run_plan(ddb, start, count, tokens, ps, n_pages, table, free, n_free, out)
    _same(got, want)
    assert want[4] == 0
    # giving them back restores the stack, whatever was in the entries that they came from
    used = got[2].copy()
    used[got[3]:n_free] = -3
    back = _run_plan(ddb, start, count, tokens, ps, n_pages, got[0], used, got[3], out, release=True)
    assert np.array_equal(back[2], free) and back[3] == n_free and back[4] == 0
    assert np.array_equal(back[0], got[0])


def test_plan_refuses_on_the_device():
    ddb = _ddb()
    ps, columns = 16, 4
    start, count = [0, -1, 5, 60, 8, 2**31 - 8], [10, 3, 70, 5, -2, 8]
    n_pages, table, free, n_free = _plan_state([0] * 6, count, 20, ps, columns, 0, 2)
    want = ref.plan(start, count, 20, ps, n_pages, free, n_free, table)
    assert want[4] == -3 and (want[1][0, :10] >= 0).all() and (want[1][1:] == -1).all()
    _same(_run_plan(ddb, start, count, 20, ps, n_pages, table, free, n_free), want)
    # too few pages: all or nothing
    start, count = [0, 0], [40, 40]
    n_pages, table, free, n_free = _plan_state(start, count, 40, ps, columns, 0, 3)
    for have in (5, 0):
        want = ref.plan(start, count, 40, ps, n_pages, free, have, table)
        assert want[4] == -7
        _same(_run_plan(ddb, start, count, 40, ps, n_pages, table, free, have), want)
    _same(_run_plan(ddb, start, count, 40, ps, n_pages, table, free, 6), ref.plan(start, count, 40, ps, n_pages, free, 6, table))
    # a pool word out of range; page ids out of range; a full stack
    for have in (-1, n_pages + 1):
        _same(_run_plan(ddb, start, count, 40, ps, n_pages, table, free, have),
              ref.plan(start, count, 40, ps, n_pages, free, have, table))
    bad = free.copy()
    bad[n_free - 2] = n_pages
    want = ref.plan(start, count, 40, ps, n_pages, bad, n_free, table)
    assert want[4] == -1 and (want[1][0, 16:32] == -1).all()
    _same(_run_plan(ddb, start, count, 40, ps, n_pages, table, bad, n_free), want)
    got = _run_plan(ddb, start, count, 40, ps, n_pages, table, free, n_free, release=True)
    assert got[3] == n_free and got[4] == -7 and np.array_equal(got[2], free)


def test_plan_unaligned_slots_and_no_token_columns():
    ddb = _ddb()
    start, count, tokens, ps = [3, 40, 0], [21, 0, 13], 21, 16
    n_pages, table, free, n_free = _plan_state(start, count, tokens, ps, 4, 0, 5)
    want = ref.plan(start, count, tokens, ps, n_pages, free, n_free, table)
    t, p, err = _i32(table), _i32([n_free, 0]), _i32([0])
    buf = torch.full((3 * tokens + 2,), -9, dtype=torch.int32, device=DEV)
    slots = buf[1:1 + 3 * tokens].view(3, tokens)                       # rows off 16-byte boundaries
    ddb.llama_paged_plan(_i32(start), _i32(count), ps, n_pages, _i32(free), p, t, slots, err_dev=err)
    assert np.array_equal(slots.cpu().numpy(), want[1]) and np.array_equal(t.cpu().numpy(), want[0])
    assert buf[0] == -9 and buf[-1] == -9 and p.tolist() == [want[3], 0]
    # no token columns: a count above 0 is out of range, nothing is taken
    none = torch.empty(3, 0, dtype=torch.int32, device=DEV)
    p, t = _i32([n_free, 0]), _i32(table)
    ddb.llama_paged_plan(_i32(start), _i32([0, 0, 0]), ps, n_pages, _i32(free), p, t, none, err_dev=err)
    assert p.tolist() == [n_free, 0] and int(err[0]) == 0
    ddb.llama_paged_plan(_i32(start), _i32(count), ps, n_pages, _i32(free), p, t, none, err_dev=err)
    assert p.tolist() == [n_free, 0] and int(err[0]) == -3 and np.array_equal(t.cpu().numpy(), table)
    # an empty batch passes the count on
    out = _i32([-5, 0])
    ddb.llama_paged_plan(_i32([]), _i32([]), ps, n_pages, _i32(free), p, t, torch.empty(0, 4, dtype=torch.int32, device=DEV),
                         pool_out=out)
    assert out.tolist() == [n_free, 0]


def test_plan_replayed_as_a_graph_in_place():
    """64 replays of a captured one-token plan whose lengths the graph advances."""
    ddb = _ddb()
    B, ps, columns, steps = 5, 16, 8, 64
    n_pages, table, free, n_free = _plan_state([0] * B, None, 1, ps, columns, 0, 4)
    start, count = _i32([0, 3, 15, 16, 40]), _i32([1, 1, 0, 1, 1])
    t, f, p, err = _i32(table), _i32(free), _i32([n_free, 0]), _i32([0])
    held = [0, 1, 1, 1, 3]
    for b, h in enumerate(held):     # what `start` holds already
        for j in range(h):
            t[b, j] = 1000 % n_pages
    slots = torch.empty(B, 1, dtype=torch.int32, device=DEV)
    t0, p0 = t.clone(), p.clone()

    def step():
        ddb.llama_paged_plan(start, count, ps, n_pages, f, p, t, slots, err_dev=err)
        start.add_(count)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    start.copy_(_i32([0, 3, 15, 16, 40]))
    t.copy_(t0)
    p.copy_(p0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    s, tab, fr, n = [0, 3, 15, 16, 40], t0.cpu().numpy(), free, n_free
    for _ in range(steps):
        graph.replay()
        torch.cuda.synchronize()
        tab, want, fr, n, e = ref.plan(s, [1, 1, 0, 1, 1], 1, ps, n_pages, fr, n, tab)
        assert e == 0 and np.array_equal(slots.cpu().numpy(), want) and p.tolist() == [n, 0]
        s = [a + c for a, c in zip(s, [1, 1, 0, 1, 1])]
    assert np.array_equal(t.cpu().numpy(), tab) and int(err[0]) == 0


# ----------------------------------------------------------------------------- store

@pytest.mark.parametrize("dtype,heads,dim", [(torch.bfloat16, 8, 128), (torch.bfloat16, 1, 128), (torch.float32, 2, 64),
                                             (torch.float32, 3, 32), (torch.float32, 1, 128)])
@pytest.mark.parametrize("batch,tokens,src_seq,src_pos,ps", [(1, 1, 1, 0, 16), (3, 37, 50, 13, 16), (5, 130, 130, 0, 64),
                                                            (2, 1025, 1100, 75, 1024)])
def test_store(dtype, heads, dim, batch, tokens, src_seq, src_pos, ps):
    ddb = _ddb()
    gen = torch.Generator().manual_seed(tokens)
    n_pages = batch * ref.ceil_div(tokens, ps) + 2
    k, v = (torch.randn(batch, heads, src_seq, dim, generator=gen).to(dtype) for _ in range(2))
    pk, pv = (torch.randn(n_pages, heads, ps, dim, generator=gen).to(dtype) for _ in range(2))
    slots = torch.randperm(n_pages * ps, generator=gen)[:batch * tokens].view(batch, tokens).to(torch.int32)
    slots[torch.rand(batch, tokens, generator=gen) < 0.2] = -1
    wk, wv = pk.clone(), pv.clone()
    for b in range(batch):
        for t in range(tokens):
            s = int(slots[b, t])
            if s >= 0:
                wk[s // ps, :, s % ps] = k[b, :, src_pos + t]
                wv[s // ps, :, s % ps] = v[b, :, src_pos + t]
    kv = ddb.PagedCache(pk.to(DEV), pv.to(DEV))
    err = _i32([0])
    ddb.llama_paged_store(k.to(DEV), v.to(DEV), slots.to(DEV), kv, src_pos, err_dev=err)
    assert torch.equal(kv.k.cpu(), wk) and torch.equal(kv.v.cpu(), wv) and int(err[0]) == 0
    # a slot behind the cache and negative ones are skipped, the first recorded
    over = torch.tensor([[n_pages * ps], [-2 ** 31], [2 ** 31 - 1]], dtype=torch.int32)[:batch]
    ddb.llama_paged_store(k.to(DEV), v.to(DEV), over.to(DEV), kv, src_pos, err_dev=err)
    assert torch.equal(kv.k.cpu(), wk) and torch.equal(kv.v.cpu(), wv) and int(err[0]) == -1


# ----------------------------------------------------------------------------- attention

def _paged(lens, heads, dim, ps, dtype, seed, scale=1.0):
    """Random K, V of `lens` positions in pages of random order; everything that no
    length covers is NaN, table entries behind the length are garbage."""
    gen = torch.Generator().manual_seed(seed)
    n = [max(0, x) for x in lens]
    need = [ref.ceil_div(x, ps) for x in n]
    n_pages, columns = sum(need) + 2, max(need) + 2
    perm = torch.randperm(n_pages, generator=gen)
    pk, pv = (torch.full((n_pages, heads, ps, dim), float("nan")) for _ in range(2))
    table = torch.randint(-2 ** 31, 2 ** 31 - 1, (len(lens), columns), generator=gen).to(torch.int32)
    rows, used = [], 0
    for b, (x, c) in enumerate(zip(n, need)):
        k, v = (torch.randn(heads, x, dim, generator=gen) * scale for _ in range(2))
        k, v = k.to(dtype).float(), v.to(dtype).float()
        rows.append((k, v))
        for j in range(c):
            page = int(perm[used])
            used += 1
            table[b, j] = page
            part = slice(j * ps, min(x, (j + 1) * ps))
            pk[page, :, :part.stop - part.start] = k[:, part]
            pv[page, :, :part.stop - part.start] = v[:, part]
    return rows, pk.to(dtype).to(DEV), pv.to(dtype).to(DEV), table.to(DEV)


def _attend(ddb, q, kv, table, lens, max_len, err=None):
    need = ddb.llama_paged_attention_workspace_bytes(q.shape[0], q.shape[1], kv.n_kv_heads, kv.head_dim, max_len)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    o = torch.full_like(q, float("nan"))
    ddb.llama_paged_attention(q, kv, table, _i32(lens), max_len, o, ws, err_dev=err)
    return o


SHAPES = {  # dtype, query heads, KV heads, head size
    "8b": (torch.bfloat16, 32, 8, 128), "70b": (torch.bfloat16, 64, 8, 128), "mha": (torch.bfloat16, 4, 4, 128),
    "mqa8": (torch.bfloat16, 8, 1, 128), "group2": (torch.bfloat16, 6, 3, 128),
    "group3": (torch.bfloat16, 6, 2, 128), "group16": (torch.bfloat16, 16, 1, 128), "group64": (torch.bfloat16, 64, 1, 128),
    "f32-64": (torch.float32, 4, 2, 64), "f32-32": (torch.float32, 6, 2, 32), "f32-128": (torch.float32, 8, 8, 128),
    "f32-group64": (torch.float32, 64, 1, 128),
}
LENS = {
    "one": [1], "short": [1, 16, 0, 17, 127], "chunk": [128, 129, 0, 255, 256, 257], "empty": [0, 0],
    "long": [5000, 1, 0, 2049], "page-end": [64, 63, 65, 1024, 1023, 1025],
}


@pytest.mark.parametrize("ps", [16, 64, 1024])
@pytest.mark.parametrize("case", LENS)
@pytest.mark.parametrize("shape", SHAPES)
def test_attention_matches_reference(shape, case, ps):
    ddb = _ddb()
    dtype, Hq, Hkv, D = SHAPES[shape]
    lens = LENS[case]
    rows, pk, pv, table = _paged(lens, Hkv, D, ps, dtype, 7)
    q = torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(3)).to(dtype)
    err = _i32([0])
    o = _attend(ddb, q.to(DEV), ddb.PagedCache(pk, pv), table, lens, max(max(lens), 1), err=err)
    got = o.double().cpu().numpy()
    assert int(err[0]) == 0
    for b, x in enumerate(lens):
        k, v = (t.double().numpy() for t in rows[b])
        want, mass, reach = ref.attention(q[b].double().numpy(), k, v)
        tol = ref.attention_tol(want, mass, reach, "bf16" if dtype is torch.bfloat16 else "f32", D, x)
        assert np.all(np.isfinite(got[b])), f"sequence {b} of {x} keys"
        assert np.all(np.abs(got[b] - want) <= tol), f"sequence {b} of {x} keys: {np.max(np.abs(got[b] - want) - tol)}"


def test_pages_beyond_32_bit_offsets():
    """A cache of 2.3e9 elements each for K and V: rows stored to, attended in and moved between pages at its
    end give what a small cache gives."""
    ddb = _ddb()
    H, D, ps, n = 8, 128, 16, 140000
    assert n * H * ps * D > 2 ** 31
    gen = torch.Generator().manual_seed(5)
    L, B = 150, 2
    k, v = (torch.randn(B, H, L, D, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2))
    q = torch.randn(B, 32, D, generator=gen).to(torch.bfloat16).to(DEV)
    columns = 11
    near = torch.arange(B * columns).view(B, columns)
    out = []
    for n_pages, table in ((B * columns, near), (n, n - 1 - near)):
        pk = torch.zeros(n_pages, H, ps, D, dtype=torch.bfloat16, device=DEV)
        kv = ddb.PagedCache(pk, torch.zeros_like(pk))
        t = torch.arange(L)
        slots = (table[:, t // ps] * ps + t % ps).to(torch.int32).contiguous().to(DEV)
        tab, err = table.to(torch.int32).contiguous().to(DEV), _i32([0])
        ddb.llama_paged_store(k, v, slots, kv, err_dev=err)
        o = _attend(ddb, q, kv, tab, [L, L], L, err=err)
        ddb.llama_beam_reorder(_i32([1, 0]), 2, _i32([L, L]), tab, ddb.PagedCacheList([kv]), err_dev=err)
        o2 = _attend(ddb, q, kv, tab, [L, L], L, err=err)
        assert int(err[0]) == 0
        out.append((o, o2, tab.cpu()))
        del pk, kv
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    assert not torch.equal(out[0][0], out[0][1]) and torch.equal(out[0][2], (n - 1 - out[1][2]).to(torch.int32))


def test_attention_with_an_error_on_record():
    """An error word that an earlier call set changes nothing."""
    ddb = _ddb()
    _, pk, pv, table = _paged([700, 20], 8, 128, 16, torch.bfloat16, 13)
    kv = ddb.PagedCache(pk, pv)
    q = torch.randn(2, 32, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    err = _i32([-7])
    assert torch.equal(_attend(ddb, q, kv, table, [700, 20], 700, err=err), _attend(ddb, q, kv, table, [700, 20], 700))
    assert int(err[0]) == -7


def test_attention_wide_scores():
    """Scores far apart (one key takes all the weight) and equal ones."""
    ddb = _ddb()
    lens = [700, 300]
    rows, pk, pv, table = _paged(lens, 8, 128, 16, torch.bfloat16, 5, scale=8.0)
    q = (torch.randn(2, 32, 128, generator=torch.Generator().manual_seed(4)) * 8).to(torch.bfloat16)
    q[1] = 0
    got = _attend(ddb, q.to(DEV), ddb.PagedCache(pk, pv), table, lens, 700).double().cpu().numpy()
    for b, x in enumerate(lens):
        k, v = (t.double().numpy() for t in rows[b])
        want, mass, reach = ref.attention(q[b].double().numpy(), k, v)
        assert np.all(np.abs(got[b] - want) <= ref.attention_tol(want, mass, reach, "bf16", 128, x))


@pytest.mark.parametrize("shape", ["8b", "group3", "f32-64"])
def test_attention_bad_lengths_and_pages(shape):
    """Lengths out of range give rows of zeros, bad page ids leave their own row undefined; both are
    recorded and the other rows are what they are without them."""
    ddb = _ddb()
    dtype, Hq, Hkv, D = SHAPES[shape]
    lens = [40, 300, 200, 129]
    _, pk, pv, table = _paged(lens, Hkv, D, 16, dtype, 8)
    kv = ddb.PagedCache(pk, pv)
    q = torch.randn(4, Hq, D, generator=torch.Generator().manual_seed(6)).to(dtype).to(DEV)
    good = _attend(ddb, q, kv, table, lens, 300)
    for bad in (-1, 301, 2 ** 31 - 1, -2 ** 31):
        err = _i32([0])
        o = _attend(ddb, q, kv, table, [40, bad, 200, 129], 300, err=err)
        assert int(err[0]) == -3 and torch.equal(o[[0, 2, 3]], good[[0, 2, 3]]) and not o[1].any()
    # the table row bounds the length too
    err = _i32([0])
    o = _attend(ddb, q, kv, table[:, :10].contiguous(), lens, 300, err=err)
    assert int(err[0]) == -3 and torch.equal(o[[0, 3]], good[[0, 3]]) and not o[1:3].any()
    for page in (-1, kv.n_pages, 2 ** 31 - 1, -2 ** 31):
        bad = table.clone()
        bad[2, 3] = page
        err = _i32([0])
        o = _attend(ddb, q, kv, bad, lens, 300, err=err)
        assert int(err[0]) == -1 and torch.equal(o[[0, 1, 3]], good[[0, 1, 3]])
    torch.cuda.synchronize()


@pytest.mark.parametrize("shape", ["8b", "group3", "f32-64"])
def test_attention_does_not_depend_on_batch_pages_or_split(shape):
    """A sequence alone, in a batch of 1100, on other page sizes and under another bound: the same bits."""
    ddb = _ddb()
    dtype, Hq, Hkv, D = SHAPES[shape]
    lens = [(37 * i) % 290 for i in range(1100)]
    rows, pk, pv, table = _paged(lens, Hkv, D, 16, dtype, 9)
    q = torch.randn(1100, Hq, D, generator=torch.Generator().manual_seed(2)).to(dtype).to(DEV)
    kv = ddb.PagedCache(pk, pv)
    o = _attend(ddb, q, kv, table, lens, 290)
    for b in (0, 3, 17, 1023, 1024, 1099):
        alone = _attend(ddb, q[b:b + 1].contiguous(), kv, table[b:b + 1].contiguous(), lens[b:b + 1], 4000)
        assert torch.equal(alone[0], o[b])
        ps = 128
        k = torch.zeros(3, Hkv, ps, D, dtype=dtype)
        v = torch.zeros_like(k)
        for j in range(3):
            part = slice(j * ps, min(lens[b], (j + 1) * ps))
            if part.stop > part.start:
                k[j, :, :part.stop - part.start] = rows[b][0][:, part].to(dtype)
                v[j, :, :part.stop - part.start] = rows[b][1][:, part].to(dtype)
        other = _attend(ddb, q[b:b + 1].contiguous(), ddb.PagedCache(k.to(DEV), v.to(DEV)), _i32([[0, 1, 2]]),
                        lens[b:b + 1], 300)
        assert torch.equal(other[0], o[b])


def test_attention_on_another_stream_and_in_graphs():
    """Two captured graphs that share a workspace, replayed in turn, and a call on a side stream."""
    ddb = _ddb()
    lens = [900, 33]
    _, pk, pv, table = _paged(lens, 8, 128, 16, torch.bfloat16, 11)
    kv = ddb.PagedCache(pk, pv)
    q = [torch.randn(2, 32, 128, generator=torch.Generator().manual_seed(s)).to(torch.bfloat16).to(DEV) for s in (1, 2)]
    want = [_attend(ddb, x, kv, table, lens, 900) for x in q]
    ws = torch.empty(ddb.llama_paged_attention_workspace_bytes(2, 32, 8, 128, 900), dtype=torch.uint8, device=DEV)
    ln, outs, graphs = _i32(lens), [torch.empty_like(x) for x in q], []
    torch.cuda.synchronize()
    for x, o in zip(q, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ddb.llama_paged_attention(x, kv, table, ln, 900, o, ws)
        graphs.append(graph)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o = _attend(ddb, q[0], kv, table, lens, 900)
    side.synchronize()
    assert torch.equal(o, want[0])


# ----------------------------------------------------------------------------- the block's decode step

@pytest.mark.parametrize("dims", [workloads.BlockDims(512, 8, 2, 128, 1024), workloads.BlockDims(1024, 8, 1, 128, 512),
                                  workloads.BlockDims(256, 2, 2, 128, 256),
                                  workloads.BlockDims(1024, 96, 12, 128, 256)],
                         ids=["group4", "group8", "group1", "one-segment-qkv"])
@pytest.mark.parametrize("ps", [16, 128])
def test_paged_decode_step_equals_the_contiguous_one(dims, ps):
    """Ragged prompts prefilled, planned, stored and decoded for 20 steps on pages: y and the attention
    output equal the contiguous cache's, bit for bit; rows behind the positions stay NaN."""
    ddb = _ddb()
    B, T, max_seq, steps = 3, 130, 320, 20
    lens = [130, 1, 97]
    w, g = workloads.make_weights(dims, weight_std=0.03)
    dev = torch.device(DEV)
    blk = ddb.LlamaBlock(dims, {k: t.to(dev) for k, t in w.items()}, {k: t.to(dev) for k, t in g.items()}, max_seq)
    x = workloads.make_x(B, T, dims.d_model).to(dev)
    kc = torch.full((B, dims.n_kv_heads, max_seq, 128), float("nan"), dtype=torch.bfloat16, device=dev)
    vc = kc.clone()
    blk.prefill(x, ddb.KVCache(kc, vc), torch.empty_like(x), blk.workspace(B, T))
    columns = ref.ceil_div(max_seq, ps)
    n_pages = B * columns
    pk = torch.full((n_pages, dims.n_kv_heads, ps, 128), float("nan"), dtype=torch.bfloat16, device=dev)
    kv = ddb.PagedCache(pk, pk.clone())
    free = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(dev)
    pool, err = _i32([n_pages, 0]), _i32([0])
    table = torch.full((B, columns), -1, dtype=torch.int32, device=dev)
    slots = torch.empty(B, T, dtype=torch.int32, device=dev)
    pos = _i32(lens)
    ddb.llama_paged_plan(torch.zeros_like(pos), pos, ps, n_pages, free, pool, table, slots, err_dev=err)
    ddb.llama_paged_store(kc, vc, slots, kv, err_dev=err)
    one, step_slots = torch.ones_like(pos), torch.empty(B, 1, dtype=torch.int32, device=dev)
    ws, wp = blk.workspace(B, 1), blk.workspace(B, 1)
    for s in range(steps):
        xs = workloads.make_x(B, 1, dims.d_model, seed=50 + s).to(dev)
        y, yp = torch.empty_like(xs), torch.empty_like(xs)
        blk.decode_seqpos(xs, ddb.KVCache(kc, vc), pos, y, ws)
        ddb.llama_paged_plan(pos, one, ps, n_pages, free, pool, table, step_slots, err_dev=err)
        blk.decode_paged(xs, kv, table, pos, yp, wp)
        torch.cuda.synchronize()
        assert blk.poll_error() == 0 and int(err[0]) == 0
        assert torch.equal(y, yp), f"step {s}"
        # the step's attention alone, from its own q
        mid = blk.intermediates(wp, B, 1)
        o = _attend(ddb, mid["q"].reshape(B, dims.n_heads, 128).contiguous(), kv, table, (pos + 1).tolist(), max_seq)
        assert torch.equal(o.view(B, -1), mid["o"])
        pos.add_(1)
    rows = torch.isnan(kv.k.float()).all(dim=3).all(dim=1).sum()
    assert int(rows) == n_pages * ps - int(pos.sum())
    ddb.llama_paged_release(torch.zeros_like(pos), pos, ps, n_pages, free, pool, table, err_dev=err)
    assert pool.tolist() == [n_pages, 0] and sorted(free.tolist()) == list(range(n_pages)) and int(err[0]) == 0


@pytest.mark.parametrize("dims", [workloads.BlockDims(512, 16, 1, 128, 256), workloads.BlockDims(256, 64, 1, 128, 256),
                                  workloads.BlockDims(256, 64, 2, 128, 256)], ids=["group16", "group64", "group32"])
def test_paged_decode_step_of_wide_groups(dims):
    """Groups of more than 8 query heads, which the contiguous decode takes in a kernel of its own: the
    same bits at a position all sequences share."""
    ddb = _ddb()
    B, P, max_seq, ps = 3, 300, 320, 16
    w, g = workloads.make_weights(dims, weight_std=0.03)
    dev = torch.device(DEV)
    blk = ddb.LlamaBlock(dims, {k: t.to(dev) for k, t in w.items()}, {k: t.to(dev) for k, t in g.items()}, max_seq)
    k, v = (t.to(dev) for t in workloads.make_cache(dims, B, max_seq, P, 1))
    columns = max_seq // ps
    pk = torch.zeros(B * columns, dims.n_kv_heads, ps, 128, dtype=torch.bfloat16, device=dev)
    kv = ddb.PagedCache(pk, pk.clone())
    table = torch.randperm(B * columns, generator=torch.Generator().manual_seed(2)).view(B, columns).to(torch.int32).to(dev)
    t = torch.arange(P, device=dev)
    slots = (table[:, t // ps] * ps + t % ps).to(torch.int32).contiguous()
    ddb.llama_paged_store(k, v, slots, kv)
    x = workloads.make_x(B, 1, dims.d_model).to(dev)
    y, yp = torch.empty_like(x), torch.empty_like(x)
    blk.decode(x, ddb.KVCache(k, v), P, y, blk.workspace(B, 1))
    blk.decode_paged(x, kv, table, _i32([P] * B), yp, blk.workspace(B, 1))
    torch.cuda.synchronize()
    assert blk.poll_error() == 0 and torch.equal(y, yp)


@pytest.mark.parametrize("dtype,dims", [
    (torch.float32, workloads.TINY), (torch.float32, workloads.BlockDims(128, 4, 4, 32, 64)),
    (torch.float32, workloads.BlockDims(128, 9, 1, 128, 64)), (torch.bfloat16, workloads.BlockDims(256, 6, 2, 128, 128)),
    (torch.bfloat16, workloads.BlockDims(256, 5, 1, 128, 128)), (torch.bfloat16, workloads.BlockDims(256, 9, 1, 128, 128))],
    ids=["f32-2x64", "f32-1x32", "f32-9x128", "bf16-3x128", "bf16-5x128", "bf16-9x128"])
@pytest.mark.parametrize("P", [0, 127, 128, 700])
def test_attention_bits_equal_the_blocks_cuda_core_decode(dtype, dims, P):
    """The shapes that the tensor-core kernel does not take: the block's own decode attention, from its q."""
    ddb = _ddb()
    B, max_seq, ps = 2, 720, 16
    w, g = workloads.make_weights(dims, dtype=dtype)
    dev = torch.device(DEV)
    blk = ddb.LlamaBlock(dims, {k: t.to(dev) for k, t in w.items()}, {k: t.to(dev) for k, t in g.items()}, max_seq)
    k, v = (t.to(dev) for t in workloads.make_cache(dims, B, max_seq, P, 1, dtype=dtype))
    x = workloads.make_x(B, 1, dims.d_model, dtype=dtype).to(dev)
    ws = blk.workspace(B, 1)
    blk.decode(x, ddb.KVCache(k, v), P, torch.empty_like(x), ws)
    torch.cuda.synchronize()
    assert blk.poll_error() == 0
    mid = blk.intermediates(ws, B, 1)
    columns = max_seq // ps
    pk = torch.full((B * columns, dims.n_kv_heads, ps, dims.head_dim), float("nan"), dtype=dtype, device=dev)
    kv = ddb.PagedCache(pk, pk.clone())
    table = torch.randperm(B * columns, generator=torch.Generator().manual_seed(2)).view(B, columns).to(torch.int32).to(dev)
    t = torch.arange(P + 1, device=dev)
    ddb.llama_paged_store(k, v, (table[:, t // ps] * ps + t % ps).to(torch.int32).contiguous(), kv)
    o = _attend(ddb, mid["q"].reshape(B, dims.n_heads, dims.head_dim).contiguous(), kv, table, [P + 1] * B, max_seq)
    assert torch.equal(o.view(B, -1), mid["o"])


def test_attention_with_a_bound_far_above_the_lengths():
    """The units are counted from the lengths: a bound of a million keys changes no bit."""
    ddb = _ddb()
    for shape in ("8b", "group3", "f32-64"):
        dtype, Hq, Hkv, D = SHAPES[shape]
        lens = [200, 0, 129]
        _, pk, pv, table = _paged(lens, Hkv, D, 16, dtype, 12)
        wide = torch.full((3, 1 << 16), -1, dtype=torch.int32, device=DEV)
        wide[:, :table.shape[1]] = table
        q = torch.randn(3, Hq, D, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
        kv = ddb.PagedCache(pk, pv)
        assert torch.equal(_attend(ddb, q, kv, table, lens, 200), _attend(ddb, q, kv, wide, lens, 1 << 20))


def test_paged_decode_step_records_bad_positions_and_pages():
    ddb = _ddb()
    dims = workloads.BlockDims(512, 8, 2, 128, 1024)
    w, g = workloads.make_weights(dims)
    dev = torch.device(DEV)
    blk = ddb.LlamaBlock(dims, {k: t.to(dev) for k, t in w.items()}, {k: t.to(dev) for k, t in g.items()}, 64)
    pk = torch.zeros(8, 2, 16, 128, dtype=torch.bfloat16, device=dev)
    kv = ddb.PagedCache(pk, pk.clone())
    x = workloads.make_x(2, 1, 512).to(dev)
    y, ws = torch.empty_like(x), blk.workspace(2, 1)
    table = _i32([[0, 1, 2, 3], [4, 5, 6, 7]])
    for pos, want in (([64, 3], -3), ([-1, 3], -3), ([3, 16], -1)):
        t = table.clone()
        t[1, 1] = 8
        before = kv.k.clone()
        blk.decode_paged(x, kv, t, _i32(pos), y, ws)
        assert blk.poll_error() == want
        assert torch.equal(kv.k[[1, 2, 3, 5, 6, 7]], before[[1, 2, 3, 5, 6, 7]])
        assert blk.poll_error() == 0
    # a table row shorter than the handle's max_seq bounds the position
    blk.decode_paged(x, kv, table[:, :1].contiguous(), _i32([16, 3]), y, ws)
    assert blk.poll_error() == -3
