"""The attention of a chunk of new tokens over a paged cache against a plain 64-bit form: head layouts, lengths from one
token on, pages that end inside a tile, what lies in masked places, refusals on the device, graphs and streams."""
import numpy as np
import pytest
import torch

from tests import chunk_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def _ddb():
    import dense_decoder_block_gb300 as ddb
    ddb.lib()
    return ddb


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def make(start, count, heads, dim, ps, dtype, seed, scale=1.0):
    """Random K, V of start + count positions in pages of random order; every cache row that no sequence holds is NaN,
    table entries behind the last page are garbage.  (rows, kpages, vpages, table)"""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n = [s + c for s, c in zip(start, count)]
    need = [ref.ceil_div(x, ps) for x in n]
    n_pages, columns = sum(need) + 2, max(need) + 2
    perm = torch.randperm(n_pages, generator=gen, device=DEV)
    pk, pv = (torch.full((n_pages, heads, ps, dim), float("nan"), device=DEV, dtype=dtype) for _ in range(2))
    table = torch.randint(-2 ** 31, 2 ** 31 - 1, (len(n), columns), generator=gen, device=DEV).to(torch.int32)
    rows, used = [], 0
    for b, (x, c) in enumerate(zip(n, need)):
        k, v = ((torch.randn(heads, x, dim, generator=gen, device=DEV) * scale).to(dtype) for _ in range(2))
        rows.append((k, v))
        ids = perm[used:used + c]
        used += c
        table[b, :c] = ids.to(torch.int32)
        for pages, r in ((pk, k), (pv, v)):
            whole = torch.full((heads, c * ps, dim), float("nan"), device=DEV, dtype=dtype)
            whole[:, :x] = r
            pages[ids] = whole.view(heads, c, ps, dim).transpose(0, 1)
    return rows, pk, pv, table


def queries(batch, tokens, heads, dim, dtype, seed, count=None, scale=1.0):
    q = torch.randn(batch, tokens, heads, dim, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV) * scale
    if count is not None:
        for b, c in enumerate(count):
            q[b, max(c, 0):] = float("nan")            # padding holds anything
    return q.to(dtype)


def attend(ddb, q, kv, table, start, count, max_len, err=None, o=None, ws=None):
    need = ddb.llama_paged_chunk_attention_workspace_bytes(q.shape[0], q.shape[1], q.shape[2], kv.n_kv_heads, kv.head_dim,
                                                           max_len)
    if ws is None:
        ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    if o is None:
        o = torch.full_like(q, 7.0)
    ddb.llama_paged_chunk_attention(q, kv, table, _i32(start), _i32(count), max_len, o, ws, err_dev=err)
    return o


def check(o, q, rows, start, count, D):
    for b, (s, c) in enumerate(zip(start, count)):
        assert torch.all(o[b, c:] == 7.0), f"rows behind the {c} tokens of sequence {b} were written"
        if c == 0:
            continue
        k, v = rows[b]
        want, mass, reach = ref.chunk_attention(q[b, :c].double(), k.double(), v.double(), s)
        tol = ref.chunk_tol(want, mass, reach, q.dtype, D, s + c)
        got = o[b, :c].double()
        assert torch.isfinite(got).all(), f"sequence {b}: {c} tokens from {s}"
        over = ((got - want).abs() - tol).max()
        assert over <= 0, f"sequence {b}: {c} tokens from {s}: {float(over)} over the bound"


SHAPES = {  # type, query heads, KV heads, head size
    "8b": (BF, 32, 8, 128), "70b": (BF, 64, 8, 128), "mha": (BF, 4, 4, 128), "mqa8": (BF, 8, 1, 128), "group2": (BF, 6, 3, 128),
    "group3": (BF, 6, 2, 128), "group5": (BF, 10, 2, 128), "group16": (BF, 16, 1, 128), "group48": (BF, 48, 1, 128),
    "group64": (BF, 64, 1, 128),
    "f32-64": (F32, 4, 2, 64), "f32-32": (F32, 6, 2, 32), "f32-128": (F32, 8, 8, 128), "f32-group3": (F32, 3, 1, 64),
    "f32-group64": (F32, 64, 1, 128),
}
# start, count, tokens (columns of q)
CHUNKS = {
    "one-token": ([0, 5, 127, 128, 1000], [1, 1, 1, 1, 1], 1),
    "nothing": ([0, 40, 0], [0, 0, 0], 5),
    "first-chunk": ([0, 0, 0, 0], [16, 1, 0, 37], 37),
    "drafts": ([944, 17, 0, 255, 511], [4, 3, 4, 0, 1], 4),
    "ragged": ([0, 130, 64, 2000, 1], [200, 77, 0, 129, 256], 256),
    "page-ends": ([15, 16, 17, 63, 1023], [1, 17, 15, 65, 2], 65),
    "prompt": ([0, 700], [513, 300], 513),
    "long": ([9000], [33], 40),
}


@pytest.mark.parametrize("ps", [16, 64, 1024])
@pytest.mark.parametrize("case", CHUNKS)
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_reference(shape, case, ps):
    ddb = _ddb()
    dtype, Hq, Hkv, D = SHAPES[shape]
    start, count, tokens = CHUNKS[case]
    rows, pk, pv, table = make(start, count, Hkv, D, ps, dtype, 7)
    q = queries(len(start), tokens, Hq, D, dtype, 3, count)
    err = _i32([0])
    most = max(s + c for s, c in zip(start, count))
    o = attend(ddb, q, ddb.PagedCache(pk, pv), table, start, count, max(most, 1), err=err)
    assert int(err[0]) == 0
    check(o, q, rows, start, count, D)


@pytest.mark.parametrize("shape", ["8b", "group3", "f32-64"])
def test_many_sequences(shape):
    """More sequences than one launch maps, most of them with few tokens or none."""
    ddb = _ddb()
    dtype, Hq, Hkv, D = SHAPES[shape]
    start, count = [(37 * i) % 290 for i in range(1100)], [i % 7 if i % 3 else 0 for i in range(1100)]
    rows, pk, pv, table = make(start, count, Hkv, D, 16, dtype, 9)
    q = queries(1100, 6, Hq, D, dtype, 2, count)
    kv = ddb.PagedCache(pk, pv)
    o = attend(ddb, q, kv, table, start, count, 300)
    few = [0, 1, 2, 5, 500, 1022, 1023, 1024, 1025, 1099]
    check(o[few], q[few], [rows[i] for i in few], [start[i] for i in few], [count[i] for i in few], D)
    # a bound far above the lengths, and the same call again: the same bits
    assert torch.equal(o, attend(ddb, q, kv, table, start, count, 300))
    wide = attend(ddb, q, kv, table, start, count, 16 * table.shape[1])
    check(wide[few], q[few], [rows[i] for i in few], [start[i] for i in few], [count[i] for i in few], D)


@pytest.mark.parametrize("shape", ["8b", "70b", "mha", "group5", "group3", "f32-64", "f32-group3"])
@pytest.mark.parametrize("seqs,spread", [(2, 700), (9, 300), (33, 90), (64, 60), (65, 60)])
def test_sequences_of_many_lengths(shape, seqs, spread):
    """Tiles that are dealt out whole by their lengths: every query row is written once, whatever the mixture."""
    ddb = _ddb()
    dtype, Hq, Hkv, D = SHAPES[shape]
    start = [(53 * i * i) % (2 * spread) for i in range(seqs)]
    count = [0 if i % 5 == 3 else spread if i % 4 == 1 else 1 + (31 * i) % spread for i in range(seqs)]
    rows, pk, pv, table = make(start, count, Hkv, D, 16, dtype, 13)
    q = queries(seqs, spread, Hq, D, dtype, 6, count)
    err = _i32([0])
    o = attend(ddb, q, ddb.PagedCache(pk, pv), table, start, count, 3 * spread, err=err)
    assert int(err[0]) == 0
    check(o, q, rows, start, count, D)


def test_positions_beyond_the_largest():
    ddb = _ddb()
    rows, pk, pv, table = make([0], [4], 1, 128, 1024, BF, 1)
    wide = torch.zeros(1, (1 << 20) + 1, dtype=torch.int32, device=DEV)
    q, err = queries(1, 4, 2, 128, BF, 2), _i32([0])
    o = attend(ddb, q, ddb.PagedCache(pk, pv), wide, [(1 << 30) - 3], [4], 2 ** 31 - 1, err=err)
    assert int(err[0]) == -3 and torch.all(o == 7.0)


@pytest.mark.parametrize("shape", ["8b", "70b", "f32-128"])
@pytest.mark.parametrize("start,count", [([20000], [100]), ([3000, 0, 100], [1000, 900, 5]), ([30000, 31], [1, 1500])])
def test_split_and_whole_tiles(shape, start, count):
    """Long caches under few rows, and mixtures of long and short sequences."""
    ddb = _ddb()
    dtype, Hq, Hkv, D = SHAPES[shape]
    rows, pk, pv, table = make(start, count, Hkv, D, 64, dtype, 17)
    q = queries(len(start), max(count), Hq, D, dtype, 4, count)
    kv = ddb.PagedCache(pk, pv)
    most = max(s + c for s, c in zip(start, count))
    o = attend(ddb, q, kv, table, start, count, most)
    check(o, q, rows, start, count, D)
    assert torch.equal(o, attend(ddb, q, kv, table, start, count, most))


@pytest.mark.parametrize("shape", ["8b", "mqa8", "f32-64"])
def test_wide_scores(shape):
    """Scores far apart (one key takes all the weight), equal ones, and maxima that fall and rise along the cache."""
    ddb = _ddb()
    dtype, Hq, Hkv, D = SHAPES[shape]
    start, count = [700, 300, 1500], [20, 130, 64]
    rows, pk, pv, table = make(start, count, Hkv, D, 16, dtype, 5, scale=8.0)
    q = queries(3, 130, Hq, D, dtype, 4, count, scale=8.0)
    q[1, :130] = 0
    o = attend(ddb, q, ddb.PagedCache(pk, pv), table, start, count, 1564)
    check(o, q, rows, start, count, D)


@pytest.mark.parametrize("shape", ["8b", "70b", "group3", "group64", "f32-64"])
@pytest.mark.parametrize("start", [0, 100, 1000])
def test_a_row_does_not_see_what_lies_behind_it(shape, start):
    """Infinities and NaN in the keys and values of later tokens of the chunk change no earlier row, and a row that sees a
    value of NaN or an infinity has it in that column alone."""
    ddb = _ddb()
    dtype, Hq, Hkv, D = SHAPES[shape]
    T = 70
    rows, pk, pv, table = make([start], [T], Hkv, D, 16, dtype, 21)
    q = queries(1, T, Hq, D, dtype, 22)
    want = attend(ddb, q, ddb.PagedCache(pk, pv), table, [start], [T], start + T)

    def poke(pages, pos, cols, value):
        pages[int(table[0, pos // 16]), :, pos % 16, cols] = value
    # keys: rows in front of the poisoned one are what they were
    for value in (float("nan"), float("inf")):
        k = pk.clone()
        poke(k, start + 41, slice(None), value)
        poke(k, start + 69, slice(None), value)
        o = attend(ddb, q, ddb.PagedCache(k, pv), table, [start], [T], start + T)
        assert torch.equal(o[0, :41], want[0, :41])
        assert not torch.isfinite(o[0, 41:].float()).all(-1).any()
    # values: rows in front are what they were; rows behind are not finite in the poisoned columns alone
    v = pv.clone()
    poke(v, start + 33, slice(5, 6), float("inf"))
    poke(v, start + 50, slice(17, 19), float("nan"))
    poke(v, start + 60, slice(5, 6), float("-inf"))
    o = attend(ddb, q, ddb.PagedCache(pk, v), table, [start], [T], start + T)
    clean = [c for c in range(D) if c not in (5, 17, 18)]
    assert torch.equal(o[0, :33], want[0, :33])
    rest = o[0, 33:][:, :, clean]
    assert torch.isfinite(rest.float()).all()
    # without the poison these positions held other values: the rest of the columns do not depend on it
    assert torch.equal(rest, want[0, 33:][:, :, clean])
    assert torch.all(o[0, 33:60, :, 5] == float("inf")) and torch.isnan(o[0, 60:, :, 5]).all()
    assert torch.isfinite(o[0, :50, :, 17:19].float()).all() and torch.isnan(o[0, 50:, :, 17:19]).all()
    # an early key that every row sees
    k = pk.clone()
    poke(k, 0, slice(None), float("nan"))
    o = attend(ddb, q, ddb.PagedCache(k, pv), table, [start], [T], start + T)
    assert torch.isnan(o).all()


@pytest.mark.parametrize("shape", ["8b", "group3", "f32-64"])
def test_bad_words_and_pages(shape):
    """Starts and counts out of range leave their rows as they were, bad page ids leave theirs undefined; both are
    recorded and the other sequences are what they are without them."""
    ddb = _ddb()
    dtype, Hq, Hkv, D = SHAPES[shape]
    start, count = [40, 300, 0, 129], [5, 33, 20, 1]
    rows, pk, pv, table = make(start, count, Hkv, D, 16, dtype, 8)
    kv = ddb.PagedCache(pk, pv)
    q = queries(4, 33, Hq, D, dtype, 6, count)
    keep = [0, 2, 3]
    for s, c in ((-1, 33), (301, 33), (300, 34), (300, -1), (2 ** 31 - 1, 33), (-2 ** 31, 33), (300, 2 ** 31 - 1)):
        err = _i32([0])
        o = attend(ddb, q, kv, table, [40, s, 0, 129], [5, c, 20, 1], 333, err=err)
        assert int(err[0]) == -3 and torch.all(o[1] == 7.0)
        check(o[keep], q[keep], [rows[i] for i in keep], [start[i] for i in keep], [count[i] for i in keep], D)
    err = _i32([0])                                  # the table row bounds the positions too
    o = attend(ddb, q, kv, table[:, :10].contiguous(), start, count, 333, err=err)
    assert int(err[0]) == -3 and torch.all(o[1] == 7.0)
    for page in (-1, kv.n_pages, 2 ** 31 - 1, -2 ** 31):
        bad = table.clone()
        bad[1, 3] = page
        err = _i32([0])
        o = attend(ddb, q, kv, bad, start, count, 333, err=err)
        assert int(err[0]) == -1
        check(o[keep], q[keep], [rows[i] for i in keep], [start[i] for i in keep], [count[i] for i in keep], D)
    # an error on record changes nothing
    err = _i32([-7])
    o = attend(ddb, q, kv, table, start, count, 333, err=err)
    assert int(err[0]) == -7
    check(o, q, rows, start, count, D)


def test_one_token_agrees_with_the_single_token_call():
    ddb = _ddb()
    start = [900, 33, 0, 128]
    rows, pk, pv, table = make(start, [1] * 4, 8, 128, 16, BF, 11)
    kv = ddb.PagedCache(pk, pv)
    q = queries(4, 1, 32, 128, BF, 12)
    o = attend(ddb, q, kv, table, start, [1] * 4, 901)
    single = torch.empty_like(q[:, 0])
    ws = torch.empty(ddb.llama_paged_attention_workspace_bytes(4, 32, 8, 128, 901), dtype=torch.uint8, device=DEV)
    ddb.llama_paged_attention(q[:, 0].contiguous(), kv, table, _i32([s + 1 for s in start]), 901, single, ws)
    for b, s in enumerate(start):
        k, v = rows[b]
        want, mass, reach = ref.chunk_attention(q[b].double(), k.double(), v.double(), s)
        tol = ref.chunk_tol(want, mass, reach, BF, 128, s + 1)
        assert torch.all((o[b, 0].double() - single[b].double()).abs() <= 2 * tol[0])


def test_graphs_and_streams():
    """Two captured graphs that share a workspace, replayed in turn with lengths that move, and a side stream."""
    ddb = _ddb()
    start, count = [3000, 33], [64, 5]
    rows, pk, pv, table = make(start, count, 8, 128, 16, BF, 11)
    kv = ddb.PagedCache(pk, pv)
    qs = [queries(2, 64, 32, 128, BF, s) for s in (1, 2)]
    want = [attend(ddb, x, kv, table, start, count, 3064) for x in qs]
    short = [attend(ddb, x, kv, table, [100, 33], [64, 0], 3064) for x in qs]
    ws = torch.empty(ddb.llama_paged_chunk_attention_workspace_bytes(2, 64, 32, 8, 128, 3064), dtype=torch.uint8, device=DEV)
    st, ct, outs, graphs = _i32(start), _i32(count), [torch.empty_like(x) for x in qs], []
    torch.cuda.synchronize()
    for x, o in zip(qs, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ddb.llama_paged_chunk_attention(x, kv, table, st, ct, 3064, o, ws)
        graphs.append(graph)
    for s, c, expect in ((start, count, want), ([100, 33], [64, 0], short), (start, count, want)):
        st.copy_(_i32(s))
        ct.copy_(_i32(c))
        for o in outs:
            o.fill_(7.0)
        for _ in range(2):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, expect))
    side = torch.cuda.Stream()
    o = torch.full_like(qs[0], 7.0)
    side.wait_stream(torch.cuda.current_stream())
    ddb.llama_paged_chunk_attention(qs[0], kv, table, st, ct, 3064, o, ws, stream=side)
    side.synchronize()
    assert torch.equal(o, want[0])


def test_two_calls_at_once():
    """A call whose tiles are split and one of whole tiles, on two streams over the same cache, a workspace each."""
    ddb = _ddb()
    calls = []
    rows, pk, pv, table = make([6000, 40], [90, 1500], 8, 128, 64, BF, 21)
    kv = ddb.PagedCache(pk, pv)
    for start, count, tokens in (([6000, 40], [90, 3], 90), ([0, 40], [0, 1500], 1500)):
        q = queries(2, tokens, 32, 128, BF, tokens, count)
        calls.append((q, _i32(start), _i32(count), attend(ddb, q, kv, table, start, count, 6090)))
    streams = [torch.cuda.Stream() for _ in calls]
    spaces = [torch.empty(ddb.llama_paged_chunk_attention_workspace_bytes(2, q.shape[1], 32, 8, 128, 6090), dtype=torch.uint8,
                          device=DEV) for q, *_ in calls]
    outs = [torch.full_like(q, 7.0) for q, *_ in calls]
    torch.cuda.synchronize()
    for _ in range(4):
        for (q, st, ct, _), o, ws, stream in zip(calls, outs, spaces, streams):
            with torch.cuda.stream(stream):
                ddb.llama_paged_chunk_attention(q, kv, table, st, ct, 6090, o, ws)
    torch.cuda.synchronize()
    for (_, _, _, want), o in zip(calls, outs):
        assert torch.equal(o, want)


def test_pages_beyond_32_bit_offsets():
    """A cache of 2.3e9 elements each for K and V: pages at its end give what a small cache gives."""
    ddb = _ddb()
    H, D, ps, n = 8, 128, 16, 140000
    assert n * H * ps * D > 2 ** 31
    start, count = [100, 0], [50, 150]
    gen = torch.Generator(device=DEV).manual_seed(5)
    k, v = (torch.randn(20, H, ps, D, generator=gen, device=DEV).to(BF) for _ in range(2))
    q = queries(2, 150, 32, D, BF, 6)
    near = torch.arange(20, device=DEV).view(2, 10)
    out = []
    for n_pages, table in ((20, near), (n, n - 1 - near)):
        pk, pv = (torch.zeros(n_pages, H, ps, D, dtype=BF, device=DEV) for _ in range(2))
        pk[table.reshape(-1)], pv[table.reshape(-1)] = k, v
        err = _i32([0])
        out.append(attend(ddb, q, ddb.PagedCache(pk, pv), table.to(torch.int32).contiguous(), start, count, 150, err=err))
        assert int(err[0]) == 0
        del pk, pv
    assert torch.equal(out[0], out[1])


@pytest.mark.parametrize("shape", ["8b", "f32-128"])
def test_follows_kernels_that_start_their_dependents_early(shape):
    """llama_rmsnorm writes every row of the pages, the attention follows at once: the result is that after a wait."""
    ddb = _ddb()
    dtype, Hq, Hkv, D = SHAPES[shape]
    start, count = [3000, 1, 2500, 0], [60, 1, 7, 64]
    columns = 49
    gen = torch.Generator(device=DEV).manual_seed(4)
    table = torch.randperm(4 * columns, generator=gen, device=DEV).view(4, columns).to(torch.int32)
    raw = [torch.randn(4 * columns, Hkv, 64, D, generator=gen, device=DEV).to(dtype) for _ in range(2)]
    gain = (torch.rand(D, generator=gen, device=DEV) + 0.5).to(dtype)
    q = queries(4, 64, Hq, D, dtype, 5)
    kv = ddb.PagedCache(torch.empty_like(raw[0]), torch.empty_like(raw[0]))

    def norm():
        for x, y in zip(raw, (kv.k, kv.v)):
            ddb.llama_rmsnorm(x, gain, y, 4 * columns * Hkv * 64, D, 1e-5)
    norm()
    torch.cuda.synchronize()
    want = attend(ddb, q, kv, table, start, count, 3100)
    for _ in range(5):
        kv.k.fill_(float("nan"))
        kv.v.fill_(float("nan"))
        norm()
        assert torch.equal(attend(ddb, q, kv, table, start, count, 3100), want)
