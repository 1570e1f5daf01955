"""What the chunk attention, the log probabilities and the sharing calls refuse before anything is launched (no GPU needed)."""
import ctypes as C

import pytest
import torch

INVALID, DIMS, WORKSPACE = -1, -2, -4
P = C.c_void_p(1 << 20)      # a 16-byte aligned address that no refused call follows
ODD = C.c_void_p((1 << 20) + 4)


@pytest.fixture(scope="module")
def lib():
    from dense_decoder_block_gb300 import _native, build
    return _native.load(build.build())


def _cache(k=P, v=P, n_pages=8, page_size=16):
    from dense_decoder_block_gb300 import _native
    return C.byref(_native.llama_paged_cache(k, v, n_pages, page_size))


def test_chunk_attention_refusals(lib):
    def attend(q=P, batch=2, tokens=5, heads=8, kv_heads=2, dim=128, dtype=1, kv=None, table=P, stride=4, start=P, count=P,
               most=64, o=P, ws=P, ws_bytes=1 << 30):
        return lib.llama_paged_chunk_attention(q, batch, tokens, heads, kv_heads, dim, dtype, kv or _cache(), table, stride,
                                               start, count, most, o, ws, ws_bytes, None, None)
    for bad in (dict(batch=-1), dict(batch=65536), dict(tokens=-1), dict(most=0), dict(most=-1), dict(stride=0), dict(q=None),
                dict(q=ODD), dict(o=None), dict(o=ODD), dict(table=None), dict(start=None), dict(count=None), dict(ws=ODD),
                dict(dtype=7), dict(kv=_cache(k=ODD)), dict(kv=_cache(n_pages=-1))):
        assert attend(**bad) == INVALID, bad
    for bad in (dict(heads=7), dict(heads=0), dict(kv_heads=0), dict(heads=130), dict(dim=64), dict(dim=80, dtype=0),
                dict(kv=_cache(page_size=20)), dict(batch=65535, tokens=40000)):
        assert attend(**bad) == DIMS, bad
    need = lib.llama_paged_chunk_attention_workspace_bytes(2, 5, 8, 2, 128, 64)
    assert need > 0 and attend(ws=None) == WORKSPACE and attend(ws_bytes=need - 1) == WORKSPACE
    assert attend(batch=0) == 0 and attend(tokens=0) == 0
    for args in ((0, 5, 8, 2, 128, 64), (2, 0, 8, 2, 128, 64), (2, 5, 8, 3, 128, 64), (2, 5, 8, 2, 100, 64),
                 (2, 5, 8, 2, 128, 0), (2, 5, 130, 2, 128, 64)):
        assert lib.llama_paged_chunk_attention_workspace_bytes(*args) == 0


def test_logprob_refusals(lib):
    def run(z=P, rows=2, vocab=100, tokens=P, n=3, lp=P, h=P, ids=P, top=P):
        return lib.llama_token_logprobs(z, rows, vocab, tokens, n, lp, h, ids, top, None, None)
    for bad in (dict(z=None), dict(rows=-1), dict(vocab=0), dict(vocab=(1 << 20) + 1), dict(n=-1), dict(n=33),
                dict(n=8, vocab=7), dict(tokens=None), dict(lp=None), dict(ids=None), dict(top=None)):
        assert run(**bad) == INVALID, bad
    assert run(rows=0) == 0


def test_fork_refusals(lib):
    from dense_decoder_block_gb300 import _native

    def fork(src=P, dst=P, lens=P, n=2, refs=P, free=P, pool=P, out=P, table=P, rows=8, stride=4, caches=None, layers=2,
             heads=2, dim=128, dtype=1, ws=P, ws_bytes=1 << 20):
        arr = (_native.llama_paged_cache * 2)(*(caches or [_native.llama_paged_cache(P, P, 8, 16)] * 2))
        return lib.llama_paged_fork(src, dst, lens, n, refs, free, pool, out, table, rows, stride, arr, layers, heads, dim,
                                    dtype, ws, ws_bytes, None, None)
    other = [_native.llama_paged_cache(P, P, 8, 16), _native.llama_paged_cache(P, P, 8, 32)]
    near = C.c_void_p((1 << 20) + 4)
    for bad in (dict(n=-1), dict(n=65536), dict(rows=0), dict(stride=0), dict(layers=0), dict(layers=129), dict(src=None),
                dict(dst=None), dict(lens=None), dict(refs=None), dict(free=None), dict(pool=None), dict(out=None),
                dict(out=near), dict(table=None), dict(caches=other), dict(heads=0), dict(dtype=3), dict(ws=ODD)):
        assert fork(**bad) == INVALID, bad
    assert fork(rows=65537) == DIMS and fork(dim=64) == DIMS
    assert lib.llama_paged_fork_workspace_bytes(2) == 32 and lib.llama_paged_fork_workspace_bytes(0) == 0
    assert fork(ws=None) == WORKSPACE and fork(ws_bytes=31) == WORKSPACE


def test_free_refusals(lib):
    def free(rows=P, lens=P, n=2, ps=16, n_pages=8, refs=P, fp=P, pool=P, out=P, table=P, t_rows=8, stride=4, ws=P,
             ws_bytes=1 << 20):
        return lib.llama_paged_free(rows, lens, n, ps, n_pages, refs, fp, pool, out, table, t_rows, stride, ws, ws_bytes, None,
                                    None)
    for bad in (dict(n=-1), dict(n=65537), dict(t_rows=0), dict(stride=-4), dict(n_pages=0), dict(rows=None), dict(lens=None),
                dict(refs=None), dict(fp=None), dict(pool=None), dict(out=None), dict(table=None), dict(ws=ODD)):
        assert free(**bad) == INVALID, bad
    for bad in (dict(ps=24), dict(t_rows=65537), dict(n=65536, stride=1 << 15)):
        assert free(**bad) == DIMS, bad
    need = lib.llama_paged_free_workspace_bytes(2, 8)
    assert need > 0 and free(ws=None) == WORKSPACE and free(ws_bytes=need - 1) == WORKSPACE
    assert lib.llama_paged_free_workspace_bytes(0, 8) == 0


def test_prefill_paged_refusals(lib):
    assert lib.llama_block_prefill_paged(None, P, 1, 4, _cache(), P, 4, P, P, P, P, 1 << 20, None) == INVALID
    assert lib.llama_block_prefill_paged_workspace_bytes(None, 1, 4) == 0


def test_python_wrappers_check_their_tensors(lib):
    import dense_decoder_block_gb300 as ddb
    z = torch.zeros(2, 10)
    with pytest.raises(ValueError):
        ddb.llama_token_logprobs(z, torch.zeros(2, dtype=torch.int32), None)
    with pytest.raises(ValueError):
        ddb.llama_token_logprobs(z[0], None, None)
    with pytest.raises(ValueError):
        ddb.llama_token_logprobs(z, None, None, top_ids=torch.zeros(2, 3, dtype=torch.int32))
