"""Forking rows of a block table and giving rows up, against plain loops."""
import numpy as np
import pytest
import torch

from tests import chunk_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _ddb():
    import dense_decoder_block_gb300 as ddb
    ddb.lib()
    return ddb


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def state(lens, rows, columns, ps, spare, seed, layers=2, heads=2, dim=128, dtype=torch.bfloat16):
    """Rows 0 .. len(lens) - 1 hold lens positions in pages of random order."""
    rng = np.random.default_rng(seed)
    need = [ref.ceil_div(n, ps) for n in lens]
    n_pages = sum(need) + spare
    order = rng.permutation(n_pages).astype(np.int32)
    table = np.full((rows, columns), -1, np.int32)
    used = 0
    for b, c in enumerate(need):
        table[b, :c] = order[used:used + c]
        used += c
    free = np.full(n_pages, -7, np.int32)
    free[:n_pages - used] = order[used:]
    gen = torch.Generator().manual_seed(seed)
    caches = [torch.randn(n_pages, heads, ps, dim, generator=gen).to(dtype) for _ in range(2 * layers)]
    return n_pages, table, free, n_pages - used, np.zeros(n_pages, np.int32), caches


class Device:
    def __init__(self, ddb, table, free, n_free, refs, caches, ps, n_ws):
        self.ddb, self.ps, self.n_pages = ddb, ps, len(refs)
        self.table, self.free, self.pool, self.refs = _i32(table), _i32(free), _i32([n_free, 0]), _i32(refs)
        self.dev = [c.to(DEV) for c in caches]
        self.caches = ddb.PagedCacheList([ddb.PagedCache(k, v) for k, v in zip(self.dev[::2], self.dev[1::2])])
        need = max(ddb.llama_paged_fork_workspace_bytes(n_ws), ddb.llama_paged_free_workspace_bytes(n_ws, self.n_pages))
        self.ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
        self.err = _i32([0])

    def fork(self, src, dst, lens, out=None):
        self.ddb.llama_paged_fork(_i32(src), _i32(dst), _i32(lens), self.refs, self.free, self.pool, self.table, self.caches,
                                  self.ws, pool_out=out, err_dev=self.err)

    def free_rows(self, rows, lens, out=None):
        self.ddb.llama_paged_free(_i32(rows), _i32(lens), self.ps, self.n_pages, self.refs, self.free, self.pool, self.table,
                                  self.ws, pool_out=out, err_dev=self.err)

    def same(self, table=None, free=None, n_free=None, refs=None, caches=None, err=0):
        if table is not None:
            assert np.array_equal(self.table.cpu().numpy(), table)
        if free is not None:
            assert np.array_equal(self.free.cpu().numpy(), free)
        if refs is not None:
            assert np.array_equal(self.refs.cpu().numpy(), refs)
        if n_free is not None:
            assert self.pool.tolist() == [n_free, 0]
        if caches is not None:
            assert all(torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8)) for a, b in zip(self.dev, caches))
        assert int(self.err) == err


def _np(caches):
    return [c.float().numpy() for c in caches]


def _t(caches, like):
    return [torch.from_numpy(c).to(o.dtype) for c, o in zip(caches, like)]


FORKS = {  # lens of the prompts, forks (src, length), page size
    "one": ([20], [(0, 20)], 16),
    "full-pages": ([32], [(0, 32), (0, 16)], 16),
    "empty": ([5, 0], [(0, 0), (1, 0)], 16),
    "many": ([100, 3, 64, 250], [(i % 4, [100, 3, 64, 250][i % 4] - i % 3) for i in range(40)], 16),
    "wide": ([3000, 1100], [(0, 3000), (1, 1100), (0, 2999), (0, 1)], 64),
    "big-pages": ([1500], [(0, 1500), (0, 1024), (0, 1023)], 1024),
}


@pytest.mark.parametrize("dtype,heads,dim", [(torch.bfloat16, 8, 128), (torch.float32, 3, 32), (torch.float32, 1, 128)])
@pytest.mark.parametrize("name", FORKS)
@pytest.mark.parametrize("out", [False, True], ids=["in-place", "pool-out"])
def test_fork_then_free(name, out, dtype, heads, dim):
    ddb = _ddb()
    lens, forks, ps = FORKS[name]
    P, F = len(lens), len(forks)
    rng = np.random.default_rng(3)
    src, flen = [f[0] for f in forks], [f[1] for f in forks]
    dst = (P + rng.permutation(F + 3)[:F]).tolist()
    n_pages, table, free, n_free, refs, caches = state(lens, P + F + 3, ref.ceil_div(max(lens), ps) + 2, ps, F + 2, 1, 2, heads,
                                                       dim, dtype)
    d = Device(ddb, table, free, n_free, refs, caches, ps, F)
    pool = _i32([-5, -5]) if out else None
    d.fork(src, dst, flen, pool)
    want = ref.fork(src, dst, flen, ps, n_pages, refs, free, n_free, table, _np(caches))
    if out:
        assert d.pool.tolist() == [n_free, 0] and pool.tolist() == [want[3], 0]
        d.pool = pool
    d.same(want[1], free, want[3], want[0], _t(want[2], caches))
    # the forks' rows given up again: the stack and the counts are what they were
    d.free[want[3]:n_free] = -3
    d.free_rows(dst, flen)
    d.same(want[1], free, n_free, refs)
    # the prompts too: as a release would leave it
    d.free_rows(list(range(P)), lens)
    end = ref.free_rows(list(range(P)), lens, ps, n_pages, refs, free, n_free, want[1])
    d.same(want[1], end[1], end[2], end[0])
    f2, p2 = _i32(free), _i32([n_free, 0])
    ddb.llama_paged_release(_i32([0] * P), _i32(lens), ps, n_pages, f2, p2, d.table)
    assert torch.equal(f2, d.free) and torch.equal(p2, d.pool)


@pytest.mark.parametrize("seed", range(6))
def test_free_of_shared_pages(seed):
    """Rows that share pages, given up in any order, some of them together."""
    ddb = _ddb()
    rng = np.random.default_rng(seed)
    ps, P = 16, 6
    lens = rng.integers(1, 400, P).tolist()
    n_pages, table, free, n_free, refs, caches = state(lens, 40, 30, ps, 60, seed, layers=1)
    d = Device(ddb, table, free, n_free, refs, caches, ps, 40)
    src = rng.integers(0, P, 20).tolist()
    flen = [int(rng.integers(0, lens[s] + 1)) for s in src]
    dst = (P + rng.permutation(34)[:20]).tolist()
    d.fork(src, dst, flen)
    refs, table, _, n_free, err = ref.fork(src, dst, flen, ps, n_pages, refs, free, n_free, table, _np(caches))
    assert err == 0
    d.same(table, free, n_free, refs)
    rows, ln = list(range(P)) + dst, lens + flen
    order = rng.permutation(len(rows))
    for part in np.array_split(order, 4):
        r, n = [rows[i] for i in part], [ln[i] for i in part]
        refs, free, n_free, err = ref.free_rows(r, n, ps, n_pages, refs, free, n_free, table)
        assert err == 0
        d.free_rows(r, n)
        d.same(table, free, n_free, refs)
    assert n_free == n_pages and not refs.any()


def test_free_of_many_entries():
    """More entries than one CTA takes: 300 rows of up to 200 pages, half of them shared."""
    ddb = _ddb()
    rng = np.random.default_rng(9)
    ps, P = 16, 150
    lens = rng.integers(0, 3200, P).tolist()
    n_pages, table, free, n_free, refs, caches = state(lens, 300, 210, ps, 200, 9, layers=1, heads=1)
    d = Device(ddb, table, free, n_free, refs, caches, ps, 300)
    src, dst = list(range(P)), (P + rng.permutation(P)).tolist()
    d.fork(src, dst, lens)
    refs, table, _, n_free, err = ref.fork(src, dst, lens, ps, n_pages, refs, free, n_free, table, [])
    d.same(table, free, n_free, refs)
    rows = list(range(P)) + dst
    ln = lens + lens
    order = rng.permutation(300)[:290]
    r, n = [rows[i] for i in order], [ln[i] for i in order]
    # (the plain loop's counts by numpy: a row per list entry)
    entries = np.concatenate([table[x, :ref.ceil_div(c, ps)] for x, c in zip(r, n)])
    drops = np.bincount(entries, minlength=n_pages)
    last = np.full(n_pages, -1)
    last[entries] = np.arange(len(entries))
    back = entries[(last[entries] == np.arange(len(entries))) & (drops[entries] > refs[entries])]
    free[n_free:n_free + len(back)] = back[::-1]
    d.free_rows(r, n)
    d.same(table, free, n_free + len(back), np.maximum(refs - drops, 0))


def test_fork_refuses_on_the_device():
    ddb = _ddb()
    ps, lens = 16, [40, 20, 33]
    n_pages, table, free, n_free, refs, caches = state(lens, 12, 5, ps, 4, 2)

    def run(src, dst, flen, err, table=table, free=free, n_free=n_free):
        d = Device(ddb, table, free, n_free, refs, caches, ps, len(src))
        d.fork(src, dst, flen)
        want = ref.fork(src, dst, flen, ps, n_pages, refs, free, n_free, table, _np(caches))
        assert want[4] == err
        d.same(want[1], free, want[3], want[0], _t(want[2], caches), err)
        return want
    # rows outside the table; a destination twice; a destination that is a source; a row onto itself
    run([0, -1, 12, 1, 2], [3, 4, 5, -1, 12], [40, 20, 20, 20, 33], -1)
    run([0, 1, 2, 1], [3, 4, 3, 5], [40, 20, 33, 20], -1)
    run([0, 3, 1], [3, 4, 5], [40, 20, 20], -1)
    run([0, 1], [0, 4], [40, 20], -1)
    # lengths
    run([0, 1, 2], [3, 4, 5], [-1, 20, 81], -3)
    run([0, 1], [3, 4], [2 ** 31 - 1, 5], -3)
    # too few pages: nothing; a pool word out of range
    run([0, 1, 2], [3, 4, 5], [40, 20, 33], -7, n_free=2)
    run([0, 1], [3, 4], [40, 20], -1, n_free=n_pages + 1)
    run([0, 1], [3, 4], [40, 20], -1, n_free=-1)
    # entries that are no page: shared ones, the unfilled one, one on the stack
    for row, col, page in ((0, 0, -1), (0, 2, n_pages), (1, 1, -2 ** 31), (1, 0, 2 ** 31 - 1)):
        bad = table.copy()
        bad[row, col] = page
        run([0, 1], [3, 4], [40, 20], -1, table=bad)
    bad = free.copy()
    bad[n_free - 1] = n_pages
    run([0, 1], [3, 4], [40, 20], -1, free=bad)


def test_free_refuses_on_the_device():
    ddb = _ddb()
    ps, lens = 16, [40, 20, 33]
    n_pages, table, free, n_free, refs, caches = state(lens, 12, 5, ps, 4, 2, layers=1)

    def run(rows, ln, err, table=table, refs=refs, n_free=n_free):
        d = Device(ddb, table, free, n_free, refs, caches, ps, len(rows))
        d.free_rows(rows, ln)
        want = ref.free_rows(rows, ln, ps, n_pages, refs, free, n_free, table)
        assert want[3] == err
        d.same(table, want[1], want[2], want[0], err=err)
    run([0, -1, 12], [40, 5, 5], -1)
    run([0, 1, 0], [40, 20, 40], -1)                       # listed twice: left out, both times
    run([0, 1, 2], [81, -1, 33], -3)
    twice = table.copy()
    twice[2, :2] = twice[1, :2]                            # given up more often than held: once
    run([1, 2], [20, 20], -1, table=twice)
    held = refs.copy()
    held[twice[1, 0]] = 1
    run([1, 2], [20, 20], -1, table=twice, refs=held)
    bad = table.copy()
    bad[0, 1] = n_pages
    run([0, 1], [40, 20], -1, table=bad)
    run([0, 1, 2], [40, 20, 33], -7, n_free=n_pages - 3)   # no room: nothing
    run([0, 1], [40, 20], -1, n_free=n_pages + 1)
    run([], [], 0)


def test_graph_of_a_round():
    """A fork and the end of its rows, captured and replayed: each replay starts and ends with the same pool."""
    ddb = _ddb()
    ps, lens = 16, [100, 47]
    n_pages, table, free, n_free, refs, caches = state(lens, 12, 10, ps, 10, 4)
    d = Device(ddb, table, free, n_free, refs, caches, ps, 8)
    src, dst, flen = _i32([0, 0, 1, 1]), _i32([5, 2, 7, 3]), _i32([100, 90, 47, 48])

    def step():
        ddb.llama_paged_fork(src, dst, flen, d.refs, d.free, d.pool, d.table, d.caches, d.ws, err_dev=d.err)
        ddb.llama_paged_free(dst, flen, ps, n_pages, d.refs, d.free, d.pool, d.table, d.ws, err_dev=d.err)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    want = ref.fork([0, 0, 1, 1], [5, 2, 7, 3], [100, 90, 47, 48], ps, n_pages, refs, free, n_free, table, _np(caches))
    d.same(want[1], free, n_free, refs, _t(want[2], caches))
