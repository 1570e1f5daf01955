"""Beam search's selection and reordering on the GPU against plain references (tests/paged_ref.py)."""
import numpy as np
import pytest
import torch

from tests import paged_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
V8B = 128256


def _ddb():
    import dense_decoder_block_gb300 as ddb
    ddb.lib()
    return ddb


def _select(ddb, logits, scores, beams, n_out, last=None, eos=-1):
    G = logits.shape[0] // beams
    need = ddb.llama_beam_select_workspace_bytes(G, beams, logits.shape[1], n_out)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    parents, tokens = (torch.full((G, n_out), -5, dtype=torch.int32, device=DEV) for _ in range(2))
    best = torch.full((G, n_out), float("nan"), device=DEV)
    ddb.llama_beam_select(logits.to(DEV), scores.to(DEV), beams, n_out, parents, tokens, best, ws,
                          last=None if last is None else last.to(DEV), eos=eos)
    return parents.cpu().numpy(), tokens.cpu().numpy(), best.cpu().numpy()


def _check(ddb, logits, scores, beams, n_out, last=None, eos=-1):
    """Parents and tokens equal; scores within the fp32 sums' error: a slice's sum of at most 8192 terms
    in (0, 1], each with a rounded difference (2^-24 of at most 2^7 where a term counts), a rounded product
    and an exponential of relative error 2^-22, added in at most 32 + 5 + 8 roundings -- below 2^-16 in the
    logarithm -- and one rounding of the score."""
    got = _select(ddb, logits, scores, beams, n_out, last, eos)
    want = ref.beam_select(logits.double().numpy(), scores.double().numpy(), beams, n_out,
                           None if last is None else last.numpy(), eos)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    fin = np.isfinite(want[2])
    assert np.array_equal(fin, np.isfinite(got[2])) and np.all(got[2][~fin] == -np.inf)
    assert np.all(np.abs(got[2][fin] - want[2][fin]) <= 2.0 ** -16 + 2.0 ** -24 * np.abs(want[2][fin]))
    return got


def _draw(rows, vocab, seed, spread=3.0):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(rows, vocab, generator=gen) * spread, -10.0 * torch.rand(rows, generator=gen)


@pytest.mark.parametrize("groups,beams,vocab,n_out", [
    (1, 1, 1, 1), (2, 3, 7, 7), (1, 4, 1000, 4), (3, 5, 1001, 10), (2, 32, 8191, 64), (1, 32, 8193, 64), (4, 8, 8192, 1),
    (1, 4, V8B, 8), (8, 4, V8B, 8), (2, 2, 1 << 20, 64), (1, 1, 64, 64), (300, 2, 130, 3)])
def test_select_matches_reference(groups, beams, vocab, n_out):
    ddb = _ddb()
    logits, scores = _draw(groups * beams, vocab, vocab + beams)
    _check(ddb, logits, scores, beams, n_out)


@pytest.mark.parametrize("vocab", [50, 1003, 20000])
def test_select_ties(vocab):
    """Many equal logits, zeros of both signs, equal rows with equal scores, all logits equal."""
    ddb = _ddb()
    logits, scores = _draw(12, vocab, 3)
    logits = torch.round(logits)
    logits[logits == 0] *= -1
    logits[1], scores[1] = logits[0], scores[0]
    logits[5] = 0.0
    logits[6], logits[7], scores[6], scores[7] = 2.5, 2.5, -1.0, -1.0
    for n_out in (1, 9, 40):
        _check(ddb, logits, scores, 4, n_out)


def test_select_first_step_ended_and_masked_beams():
    ddb = _ddb()
    V, eos = 9000, 17
    logits, scores = _draw(16, V, 5)
    last = torch.randint(0, V, (16,), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    last[last == eos] = 0
    ninf = float("-inf")
    # group 0: the first step; 1: one ended beam; 2: every beam ended; 3: an ended beam at -inf
    scores[1:4] = ninf
    last[5] = eos
    scores[5] = 0.5
    last[8:12] = eos
    last[13], scores[13] = eos, ninf
    for n_out in (4, 8, 64):
        _check(ddb, logits, scores, 4, n_out, last, eos)
    _check(ddb, logits, scores, 4, 8)                       # without last nothing has ended
    # rows whose mask leaves few tokens or none
    logits[0] = ninf
    logits[4, 3:] = ninf
    logits[6] = torch.finfo(torch.float32).min
    logits[7, :] = ninf
    logits[7, V - 1] = -3.0e38
    scores[12:] = ninf
    for n_out in (4, 64):
        _check(ddb, logits, scores, 4, n_out, last, eos)
    for e in (0, V - 1):
        last[9] = e
        _check(ddb, logits, scores, 4, 16, last, e)


@pytest.mark.parametrize("vocab", [1024, 1000])
def test_select_unaligned_logits_and_unread_rows(vocab):
    """Logits one float off a 16-byte boundary; NaN in the rows of beams that are not read."""
    ddb = _ddb()
    logits, scores = _draw(8, vocab, 11)
    scores[3] = float("-inf")
    last = torch.zeros(8, dtype=torch.int32)
    last[6] = 5
    want = ref.beam_select(logits.double().numpy(), scores.double().numpy(), 4, 8, last.numpy(), 5)
    logits[3] = float("nan")
    logits[6] = float("nan")
    buf = torch.empty(8 * vocab + 1, device=DEV)
    off = buf[1:].view(8, vocab)
    off.copy_(logits)
    for x in (off, logits):
        got = _select(ddb, x, scores, 4, 8, last, 5)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_select_in_place():
    """With as many candidates as beams the scores and last tokens may be overwritten."""
    ddb = _ddb()
    logits, scores = _draw(12, 5000, 14)
    last = torch.zeros(12, dtype=torch.int32)
    last[4] = 7
    want = _select(ddb, logits, scores, 4, 4, last, 7)
    ws = torch.empty(ddb.llama_beam_select_workspace_bytes(3, 4, 5000, 4), dtype=torch.uint8, device=DEV)
    sc, tok, par = scores.to(DEV), last.to(DEV), torch.empty(12, dtype=torch.int32, device=DEV)
    ddb.llama_beam_select(logits.to(DEV), sc, 4, 4, par, tok, sc, ws, last=tok, eos=7)
    for a, b in zip((par, tok, sc), want):
        assert np.array_equal(a.cpu().numpy().reshape(3, 4), b)


def test_select_shared_workspace_and_graphs():
    ddb = _ddb()
    logits, scores = _draw(8, 30000, 8)
    want = _select(ddb, logits, scores, 4, 8)
    ws = torch.empty(ddb.llama_beam_select_workspace_bytes(2, 4, 30000, 8), dtype=torch.uint8, device=DEV)
    pair = []
    for scale in (1.0, 2.0):
        lg, sc = (logits * scale).to(DEV), scores.to(DEV)
        out = [torch.empty(2, 8, dtype=t, device=DEV) for t in (torch.int32, torch.int32, torch.float32)]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ddb.llama_beam_select(lg, sc, 4, 8, *out, ws)
        pair.append((graph, out, lg, sc))
    for _ in range(3):
        for graph, _, _, _ in pair:
            graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(pair[0][1], want):
        assert np.array_equal(a.cpu().numpy(), b)


# ----------------------------------------------------------------------------- reorder

def _reorder(ddb, groups, beams, ps, lens, parents, layers, heads, dim, dtype, seed, mutate=None):
    gen = torch.Generator().manual_seed(seed)
    rows, columns = groups * beams, max(ref.ceil_div(max(lens), ps), 1) + 2
    n_pages = rows * columns + 1
    table = torch.randperm(n_pages, generator=gen)[:rows * columns].view(rows, columns).to(torch.int32)
    # beams share their full pages, as after an earlier call
    for g in range(groups):
        shared = lens[g * beams] // ps // 2
        table[g * beams:(g + 1) * beams, :shared] = table[g * beams, :shared]
    if mutate is not None:
        mutate(table)
    caches = [torch.randn(n_pages, heads, ps, dim, generator=gen).to(dtype) for _ in range(2 * layers)]
    dev = [c.to(DEV) for c in caches]
    tab, err = table.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    lst = ddb.PagedCacheList([ddb.PagedCache(dev[2 * i], dev[2 * i + 1]) for i in range(layers)])
    ddb.llama_beam_reorder(torch.tensor(parents, dtype=torch.int32, device=DEV), beams,
                           torch.tensor(lens, dtype=torch.int32, device=DEV), tab, lst, err_dev=err)
    want = ref.beam_reorder(table.numpy(), parents, beams, lens, ps, [c.float().numpy() for c in caches], n_pages)
    assert np.array_equal(tab.cpu().numpy(), want[0])
    for a, b in zip(dev, want[1]):
        assert np.array_equal(a.float().cpu().numpy(), b)
    assert int(err[0]) == want[2]
    return want[2]


@pytest.mark.parametrize("dtype,heads,dim", [(torch.bfloat16, 8, 128), (torch.float32, 2, 64), (torch.float32, 3, 32)])
@pytest.mark.parametrize("groups,beams,ps,length", [(1, 1, 16, 5), (1, 2, 16, 15), (2, 4, 16, 100), (3, 4, 16, 96), (2, 5, 32, 31),
                                                    (1, 8, 128, 300), (1, 16, 64, 65), (2, 32, 16, 33), (2, 3, 16, 0)])
def test_reorder_matches_reference(groups, beams, ps, length, dtype, heads, dim):
    ddb = _ddb()
    rng = np.random.default_rng(length + beams)
    maps = [rng.integers(0, beams, (groups, beams)), np.tile(np.roll(np.arange(beams), 1), (groups, 1)),
            np.tile(np.arange(beams)[::-1], (groups, 1)), np.zeros((groups, beams), int),
            np.tile(np.arange(beams), (groups, 1))]
    for i, m in enumerate(maps):
        parents = (m + beams * np.arange(groups)[:, None]).reshape(-1).tolist()
        lens = [length + 16 * g for g in range(groups) for _ in range(beams)]
        assert _reorder(ddb, groups, beams, ps, lens, parents, 1 + i % 3, heads, dim, dtype, i) == 0


def test_reorder_leaves_bad_groups_as_they_were():
    ddb = _ddb()
    args = dict(layers=2, heads=2, dim=128, dtype=torch.bfloat16, seed=1)
    lens = [20] * 6
    for parents in ([1, 0, 3, 4, 4, 3], [-1, 0, 2, 3, 4, 5], [1, 0, 2, 5, 6, 4], [2 ** 31 - 1, 0, 2, 3, 4, -2 ** 31]):
        assert _reorder(ddb, 2, 3, 16, lens, parents, **args) == -1
    assert _reorder(ddb, 2, 3, 16, [20, 20, 21, 20, 20, 20], [1, 0, 2, 3, 5, 4], **args) == -1
    assert _reorder(ddb, 2, 3, 16, [-4, -4, -4, 20, 20, 20], [1, 0, 2, 3, 5, 4], **args) == -1

    def same_page(table):
        table[1, 1] = table[0, 1]

    assert _reorder(ddb, 2, 3, 16, lens, [1, 0, 2, 3, 5, 4], mutate=same_page, **args) == -1

    def no_page(table):
        table[5, 1] = -1

    assert _reorder(ddb, 2, 3, 16, lens, [1, 0, 2, 3, 5, 4], mutate=no_page, **args) == -1
    # with no unfilled page the entry behind the full ones is not looked at
    assert _reorder(ddb, 2, 3, 16, [16] * 6, [1, 0, 2, 3, 5, 4], mutate=no_page, **args) == 0
