"""What the paged-cache and beam-search calls refuse before anything is launched (no GPU needed)."""
import ctypes as C

import pytest
import torch

INVALID, DIMS, POS, WORKSPACE = -1, -2, -3, -4
P = C.c_void_p(1 << 20)      # a 16-byte aligned address that no refused call follows
ODD = C.c_void_p((1 << 20) + 4)


@pytest.fixture(scope="module")
def lib():
    from dense_decoder_block_gb300 import _native, build
    return _native.load(build.build())


def _cache(k=P, v=P, n_pages=8, page_size=16):
    from dense_decoder_block_gb300 import _native
    return C.byref(_native.llama_paged_cache(k, v, n_pages, page_size))


def test_plan_refusals(lib):
    def plan(start=P, count=P, batch=2, tokens=3, ps=16, n_pages=8, free=P, pool=P, out=P, table=P, stride=4, slots=P):
        return lib.llama_paged_plan(start, count, batch, tokens, ps, n_pages, free, pool, out, table, stride, slots, None,
                                    None)
    for bad in (dict(batch=-1), dict(tokens=-1), dict(stride=0), dict(n_pages=0), dict(start=None), dict(count=None),
                dict(free=None), dict(pool=None), dict(out=None), dict(table=None), dict(slots=None)):
        assert plan(**bad) == INVALID, bad
    for bad in (dict(ps=0), dict(ps=8), dict(ps=24), dict(ps=2048), dict(ps=1024, n_pages=1 << 21)):
        assert plan(**bad) == DIMS, bad


def test_release_refusals(lib):
    def release(start=P, count=P, batch=2, ps=16, n_pages=8, free=P, pool=P, out=P, table=P, stride=4):
        return lib.llama_paged_release(start, count, batch, ps, n_pages, free, pool, out, table, stride, None, None)
    for bad in (dict(batch=-1), dict(stride=-4), dict(n_pages=-8), dict(start=None), dict(count=None), dict(free=None),
                dict(pool=None), dict(out=None), dict(table=None)):
        assert release(**bad) == INVALID, bad
    assert release(ps=17) == DIMS


def test_store_refusals(lib):
    def store(k=P, v=P, batch=1, tokens=4, seq=8, pos=0, slots=P, heads=2, dim=128, dtype=1, kv=None):
        return lib.llama_paged_store(k, v, batch, tokens, seq, pos, slots, heads, dim, dtype, kv or _cache(), None, None)
    for bad in (dict(batch=-1), dict(batch=65536), dict(tokens=-1), dict(pos=-1), dict(k=None), dict(v=None), dict(k=ODD),
                dict(v=ODD), dict(slots=None), dict(heads=0), dict(dtype=2), dict(kv=_cache(k=None)),
                dict(kv=_cache(v=ODD)), dict(kv=_cache(n_pages=0))):
        assert store(**bad) == INVALID, bad
    for bad in (dict(dim=64), dict(dim=96, dtype=0), dict(kv=_cache(page_size=8)), dict(heads=1 << 17),
                dict(kv=_cache(n_pages=1 << 24, page_size=64))):
        assert store(**bad) == DIMS, bad
    assert store(pos=5) == POS and store(tokens=9) == POS
    assert store(batch=0) == 0 and store(tokens=0) == 0


def test_attention_refusals(lib):
    def attend(q=P, batch=2, heads=8, kv_heads=2, dim=128, dtype=1, kv=None, table=P, stride=4, lens=P, most=64, o=P,
               ws=P, ws_bytes=1 << 30):
        return lib.llama_paged_attention(q, batch, heads, kv_heads, dim, dtype, kv or _cache(), table, stride, lens, most, o,
                                         ws, ws_bytes, None, None)
    for bad in (dict(batch=-1), dict(batch=65536), dict(most=0), dict(most=-1), dict(stride=0), dict(q=None), dict(q=ODD),
                dict(o=None), dict(o=ODD), dict(table=None), dict(lens=None), dict(ws=ODD), dict(dtype=7),
                dict(kv=_cache(k=ODD)), dict(kv=_cache(n_pages=-1))):
        assert attend(**bad) == INVALID, bad
    for bad in (dict(heads=7), dict(heads=0), dict(kv_heads=0), dict(heads=130), dict(dim=64), dict(dim=80, dtype=0),
                dict(kv=_cache(page_size=20))):
        assert attend(**bad) == DIMS, bad
    need = lib.llama_paged_attention_workspace_bytes(2, 8, 2, 128, 64)
    assert need == 2 * 8 * 132 * 4
    assert attend(ws=None) == WORKSPACE and attend(ws_bytes=need - 1) == WORKSPACE
    assert attend(batch=0) == 0
    for args in ((0, 8, 2, 128, 64), (2, 8, 3, 128, 64), (2, 8, 2, 100, 64), (2, 8, 2, 128, 0), (2, 130, 2, 128, 64)):
        assert lib.llama_paged_attention_workspace_bytes(*args) == 0
    assert lib.llama_block_decode_paged(None, P, 1, _cache(), P, 4, P, P, P, 0, None) == INVALID


def test_select_refusals(lib):
    def select(logits=P, groups=2, beams=4, vocab=100, scores=P, last=None, eos=-1, n=8, par=P, tok=P, best=P, ws=P,
               ws_bytes=1 << 30):
        return lib.llama_beam_select(logits, groups, beams, vocab, scores, last, eos, n, par, tok, best, ws, ws_bytes, None)
    for bad in (dict(groups=-1), dict(groups=20000), dict(beams=0), dict(beams=33), dict(vocab=0), dict(vocab=(1 << 20) + 1),
                dict(n=0), dict(n=65), dict(vocab=7), dict(last=P), dict(last=P, eos=100), dict(logits=None),
                dict(scores=None), dict(par=None), dict(tok=None), dict(best=None), dict(ws=ODD)):
        assert select(**bad) == INVALID, bad
    need = lib.llama_beam_select_workspace_bytes(2, 4, 100, 8)
    assert need > 0 and select(ws_bytes=need - 1) == WORKSPACE and select(ws=None) == WORKSPACE
    assert select(groups=0) == 0
    assert lib.llama_beam_select_workspace_bytes(2, 4, 7, 8) == 0


def test_reorder_refusals(lib):
    from dense_decoder_block_gb300 import _native

    def reorder(parents=P, groups=2, beams=4, lens=P, table=P, stride=4, layers=2, heads=2, dim=128, dtype=1, caches=None):
        arr = (_native.llama_paged_cache * 2)(*(caches or [_native.llama_paged_cache(P, P, 8, 16)] * 2))
        return lib.llama_beam_reorder(parents, groups, beams, lens, table, stride, arr, layers, heads, dim, dtype, None, None)
    other = [_native.llama_paged_cache(P, P, 8, 16), _native.llama_paged_cache(P, P, 9, 16)]
    for bad in (dict(groups=-1), dict(groups=65536), dict(beams=0), dict(stride=0), dict(layers=0), dict(layers=129),
                dict(parents=None), dict(lens=None), dict(table=None), dict(caches=other), dict(heads=0), dict(dtype=3)):
        assert reorder(**bad) == INVALID, bad
    assert reorder(beams=33) == DIMS and reorder(dim=64) == DIMS
    assert reorder(groups=0) == 0 and reorder(beams=1) == 0
    assert lib.llama_beam_reorder(P, 2, 4, P, P, 4, None, 2, 2, 128, 1, None, None) == INVALID


def test_python_wrappers_check_their_tensors(lib):
    import dense_decoder_block_gb300 as ddb
    cpu = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ddb.PagedCache(cpu, cpu)                       # not on a device
    with pytest.raises(ValueError):
        ddb.PagedCache(cpu, cpu[:, :1])
    with pytest.raises(ValueError):
        ddb.PagedCacheList([])
