"""Joining of tiles that the chunk attention splits over CTAs: pieces without weight, and several launches of one call."""
import numpy as np
import pytest
import torch

from tests import chunk_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
SHAPES = {"bf16": (BF, 4, 1, 128), "bf16-8b": (BF, 32, 8, 128), "f32-64": (F32, 4, 2, 64), "f32-128": (F32, 8, 8, 128)}


def _ddb():
    import dense_decoder_block_gb300 as ddb
    ddb.lib()
    return ddb


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def one_sequence(L, heads, dim, ps, dtype, gen):
    """Random K, V [heads, L, dim], and a function that lays them out in pages of random order: (cache, table)."""
    k, v = (torch.randn(heads, L, dim, generator=gen, device=DEV).to(dtype) for _ in range(2))
    n = ref.ceil_div(L, ps)
    perm = torch.randperm(n, generator=gen, device=DEV)

    def pages(ddb):
        out = []
        for rows in (k, v):
            whole = torch.zeros(heads, n * ps, dim, dtype=dtype, device=DEV)
            whole[:, :L] = rows
            p = torch.empty(n, heads, ps, dim, dtype=dtype, device=DEV)
            p[perm] = whole.view(heads, n, ps, dim).transpose(0, 1)
            out.append(p)
        return ddb.PagedCache(*out), perm.to(torch.int32)[None].contiguous()
    return k, v, pages


def attend(ddb, q, kv, table, start, count, max_len):
    ws = torch.full((ddb.llama_paged_chunk_attention_workspace_bytes(q.shape[0], q.shape[1], q.shape[2], kv.n_kv_heads,
                                                                     kv.head_dim, max_len),), 0xff, dtype=torch.uint8, device=DEV)
    o, err = torch.full_like(q, 7.0), _i32([0])
    ddb.llama_paged_chunk_attention(q, kv, table, _i32(start), _i32(count), max_len, o, ws, err_dev=err)
    assert int(err) == 0
    return o


@pytest.mark.parametrize("held,T", [(9000, 20), (300, 20), (9000, 150)], ids=["split", "whole", "split-halves"])
@pytest.mark.parametrize("shape", SHAPES)
def test_values_of_keys_without_weight(shape, held, T):
    """Keys of score -inf have weight 0, and 0 times a NaN or an infinity is NaN in that column, wherever the tile is cut: the
    first half of the cache has such keys alone (whole pieces of a split tile), with one NaN and one infinity among its values."""
    ddb = _ddb()
    dtype, Hq, Hkv, D = SHAPES[shape]
    gen = torch.Generator(device=DEV).manual_seed(3)
    k, v, pages = one_sequence(held + T, Hkv, D, 16, dtype, gen)
    half = held // 2
    k[:, :half, 0] = float("-inf")
    v[:, 100, 5], v[:, 101, 9] = float("nan"), float("inf")
    q = torch.randn(1, T, Hq, D, generator=gen, device=DEV)
    q[..., 0] = q[..., 0].abs() + 0.1
    q = q.to(dtype)
    kv, table = pages(ddb)
    o = attend(ddb, q, kv, table, [held], [T], held + T)
    assert torch.isnan(o[..., 5]).all() and torch.isnan(o[..., 9]).all()
    # the other columns are the attention over the second half
    rest = [c for c in range(D) if c not in (5, 9)]
    want, mass, reach = ref.chunk_attention(q[0].double(), k[:, half:].double(), v[:, half:].double(), held - half)
    tol = ref.chunk_tol(want, mass, reach, dtype, D, held + T)
    assert torch.isfinite(o[..., rest].float()).all()
    assert float(((o[0].double() - want).abs() - tol)[..., rest].max()) <= 0
    # keys of score -inf alone: no finite softmax
    k[:, :, 0] = float("-inf")
    kv, table = pages(ddb)
    assert torch.isnan(attend(ddb, q, kv, table, [held], [T], held + T)).all()


@pytest.mark.parametrize("shape", SHAPES)
def test_writes_no_more_than_its_workspace(shape):
    """Calls with exactly the workspace that they ask for: what lies behind it stays as it was, and so does the result beside a
    larger one."""
    ddb = _ddb()
    dtype, Hq, Hkv, D = SHAPES[shape]
    for T, held in ((1, 384), (1, 3000), (1, 60000), (5, 700), (40, 2000), (130, 9000), (600, 100)):
        gen = torch.Generator(device=DEV).manual_seed(T + held)
        k, v, pages = one_sequence(held + T, Hkv, D, 64, dtype, gen)
        q = torch.randn(1, T, Hq, D, generator=gen, device=DEV).to(dtype)
        kv, table = pages(ddb)
        need = ddb.llama_paged_chunk_attention_workspace_bytes(1, T, Hq, Hkv, D, held + T)
        room = torch.full((need + (1 << 20),), 0xa5, dtype=torch.uint8, device=DEV)
        o, err = torch.zeros_like(q), _i32([0])
        ddb.llama_paged_chunk_attention(q, kv, table, _i32([held]), _i32([T]), held + T, o, room[:need], err_dev=err)
        assert int(err) == 0 and bool((room[need:] == 0xa5).all())
        want, mass, reach = ref.chunk_attention(q[0].double(), k.double(), v.double(), held)
        assert float(((o[0].double() - want).abs() - ref.chunk_tol(want, mass, reach, dtype, D, held + T)).max()) <= 0
        wide = torch.full_like(q, 7.0)     # a bound far above the positions: more workspace, the same result up to rounding
        if held > 400:
            table = torch.cat([table, table.new_zeros(1, 5000)], 1).contiguous()
            ws = torch.empty(ddb.llama_paged_chunk_attention_workspace_bytes(1, T, Hq, Hkv, D, 1 << 18), dtype=torch.uint8, device=DEV)
            ddb.llama_paged_chunk_attention(q, kv, table, _i32([held]), _i32([T]), 1 << 18, wide, ws, err_dev=err)
            assert int(err) == 0 and torch.equal(o, wide)


@pytest.mark.parametrize("shape,seqs", [("bf16", 1100), ("bf16-8b", 2100), ("f32-64", 300), ("f32-128", 600)])
def test_several_launches_that_split(shape, seqs):
    """More sequences than a launch takes, most of them empty or short, with a long one under few tokens in the first launch and
    in the last: each launch splits and joins, over the same partials.  Equal calls give equal bits."""
    ddb = _ddb()
    dtype, Hq, Hkv, D = SHAPES[shape]
    T, ps = 6, 64
    start, count = [0] * seqs, [0] * seqs
    long = {3: (9000, 4), seqs - 2: (7000, 6)}
    short = {0: (0, 1), 7: (30, 2), seqs // 2: (300, 6), seqs - 1: (64, 5)}
    gen = torch.Generator(device=DEV).manual_seed(6)
    used = {**long, **short}
    need = {b: ref.ceil_div(s + c, ps) for b, (s, c) in used.items()}
    n_pages = sum(need.values())
    perm = torch.randperm(n_pages, generator=gen, device=DEV)
    pk, pv = (torch.full((n_pages, Hkv, ps, D), float("nan"), dtype=dtype, device=DEV) for _ in range(2))
    table = torch.full((seqs, max(need.values())), -1, dtype=torch.int32, device=DEV)
    rows, at = {}, 0
    for b, (s, c) in used.items():
        start[b], count[b] = s, c
        ids = perm[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = ids.to(torch.int32)
        rows[b] = [torch.randn(Hkv, s + c, D, generator=gen, device=DEV).to(dtype) for _ in range(2)]
        for p, x in zip((pk, pv), rows[b]):
            whole = torch.full((Hkv, need[b] * ps, D), float("nan"), dtype=dtype, device=DEV)
            whole[:, :s + c] = x
            p[ids] = whole.view(Hkv, need[b], ps, D).transpose(0, 1)
    q = torch.randn(seqs, T, Hq, D, generator=gen, device=DEV).to(dtype)
    kv = ddb.PagedCache(pk, pv)
    o = attend(ddb, q, kv, table, start, count, 9004)
    for b in range(seqs):
        if b not in used:
            continue
        s, c = used[b]
        k, v = (x.double() for x in rows[b])
        want, mass, reach = ref.chunk_attention(q[b, :c].double(), k, v, s)
        assert float(((o[b, :c].double() - want).abs() - ref.chunk_tol(want, mass, reach, dtype, D, s + c)).max()) <= 0, b
        assert torch.all(o[b, c:] == 7.0)
    off = torch.ones(seqs, dtype=torch.bool, device=DEV)
    off[list(used)] = False
    assert torch.all(o[off] == 7.0)
    for _ in range(3):
        assert torch.equal(o, attend(ddb, q, kv, table, start, count, 9004))
