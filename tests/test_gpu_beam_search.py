"""Beam search on a small stack (BeamSearch: prefill, block tables, row store, paged decode steps, selection,
reordering) against the same search run on contiguous caches with plain index copies: logits bit for bit at
every step, tokens, parents and scores equal to the 64-bit selection's."""
import numpy as np
import pytest
import torch

import workloads
from tests import paged_ref as ref
from tests.test_gpu_stack import SMALL, VOCAB, _stack_inputs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _stack(groups, max_seq, T):
    import dense_decoder_block_gb300 as ddb
    from dense_decoder_block_gb300.stack import LlamaStack
    ddb.lib()
    dev = torch.device(DEV)
    layers, w_embed, g_final, w_out, _ = _stack_inputs()
    dl = [({k: v.to(dev) for k, v in w.items()}, {k: v.to(dev) for k, v in g.items()}) for w, g in layers]
    return ddb, LlamaStack(SMALL, dl, w_embed.to(dev), g_final.to(dev), w_out.to(dev), batch=groups, max_seq=max_seq,
                           prefill_tokens=T)


class _Plain:
    """The same search with a contiguous cache per beam, copied whole when beams move."""

    def __init__(self, ddb, st, beams, max_new, eos):
        self.ddb, self.st, self.K, self.eos = ddb, st, beams, eos
        self.rows = st.batch * beams
        self.logits = torch.empty(self.rows, VOCAB, device=DEV)
        self.ws = st.blocks[0].workspace(self.rows, 1)
        self.head_ws = torch.empty(ddb.llama_lmhead_workspace_bytes(self.rows, SMALL.d_model, VOCAB), dtype=torch.uint8,
                                   device=DEV)

    def choose(self, last):
        p, t, s = ref.beam_select(self.logits.double().cpu().numpy(), self.scores.astype(np.float64), self.K, self.K, last,
                                  self.eos)
        self.parents, self.tokens, self.scores = p.reshape(-1), t.reshape(-1), s.reshape(-1).astype(np.float32)
        at = torch.tensor(self.parents, device=DEV)
        self.kv = [(k[at].clone(), v[at].clone()) for k, v in self.kv]

    def begin(self, ids):
        st = self.st
        st.prefill(ids)
        self.kv = [(c.k.repeat_interleave(self.K, 0), c.v.repeat_interleave(self.K, 0)) for c in st.caches]
        self.logits.zero_()
        self.logits[::self.K] = st.logits
        self.scores = np.full(self.rows, -np.inf, np.float32)
        self.scores[::self.K] = 0
        self.pos = torch.full((self.rows,), ids.shape[1], dtype=torch.int32, device=DEV)
        self.choose(None)

    def step(self):
        st, ddb = self.st, self.ddb
        x = torch.empty(self.rows, 1, SMALL.d_model, dtype=torch.bfloat16, device=DEV)
        y = torch.empty_like(x)
        ids = torch.tensor(self.tokens, dtype=torch.int32, device=DEV)
        ddb.llama_embed(ids, self.rows, st.w_embed, VOCAB, SMALL.d_model, x)
        for blk, (k, v) in zip(st.blocks, self.kv):
            blk.decode_seqpos(x, ddb.KVCache(k, v), self.pos, y, self.ws)
            x, y = y, x
        out = torch.empty(self.rows, dtype=torch.int32, device=DEV)
        ddb.llama_lmhead_argmax(x, self.rows, SMALL.d_model, st.g_final, st.w_out, VOCAB, SMALL.d_model, SMALL.eps, out,
                                self.logits, self.head_ws, self.head_ws.numel())
        self.pos += 1
        self.choose(self.tokens if self.eos >= 0 else None)


def _run(groups, beams, T, max_new, ps, eos=-1, seed=21, check=True):
    ddb, st = _stack(groups, T + max_new + 3, T)
    from dense_decoder_block_gb300.stack import BeamSearch
    ids = workloads.make_token_ids(groups, T, VOCAB, seed=seed).to(DEV).to(torch.int32)
    bs = BeamSearch(st, beams, max_new, eos=eos, page_size=ps)
    plain = _Plain(ddb, st, beams, max_new, eos)
    bs.begin(ids)
    plain.begin(ids)
    history = []
    for s in range(max_new):
        if s:
            bs.step()
            plain.step()
        if s:
            assert torch.equal(bs.logits, plain.logits), f"step {s}"
        assert bs.parents.tolist() == plain.parents.tolist() and bs.tokens.tolist() == plain.tokens.tolist(), f"step {s}"
        # the fp32 scores' own rounding carries over: their difference grows by one selection's error a step
        got = bs.scores.cpu().numpy()
        assert np.all(np.abs(got - plain.scores) <= (s + 1) * (2.0 ** -16 + 2.0 ** -23 * np.abs(plain.scores))), f"step {s}"
        plain.scores = got                      # the next step's selection from the same scores
        history.append((plain.parents.copy(), plain.tokens.copy()))
        assert bs.poll_error() == 0
    tokens, scores = bs.sequences()
    rows = np.arange(groups * beams)
    want = np.zeros((groups * beams, max_new), np.int64)
    for s in range(max_new - 1, -1, -1):
        want[:, s] = history[s][1][rows]
        rows = history[s][0][rows]
    assert np.array_equal(tokens.cpu().numpy().reshape(groups * beams, max_new), want)
    assert torch.equal(scores.reshape(-1), bs.scores)
    bs.end()
    assert bs.pool.tolist() == [bs.n_pages, 0] and bs.free.tolist() == list(range(bs.n_pages))
    return ids, want, history


@pytest.mark.parametrize("groups,beams,T,max_new,ps", [(2, 3, 20, 12, 16), (1, 4, 16, 20, 16), (3, 2, 37, 30, 32),
                                                       (1, 1, 5, 6, 16), (4, 8, 130, 8, 16)])
def test_beam_search_equals_the_contiguous_one(groups, beams, T, max_new, ps):
    _run(groups, beams, T, max_new, ps)


def test_beam_search_with_ended_beams():
    """An end token that the search meets: the ended beam repeats it at its score."""
    _, want, history = _run(2, 3, 20, 10, 16)
    eos = int(history[4][1][0])
    _, ended, _ = _run(2, 3, 20, 10, 16, eos=eos)
    rows = [r for r in ended if eos in r[:-1].tolist()]
    assert rows, "the end token was not met"
    for r in rows:
        first = r.tolist().index(eos)
        assert (r[first:] == eos).all()


def test_beam_search_step_as_a_graph_and_twice():
    """A captured step replayed gives the eager search's tokens; a second search reuses the pages."""
    from dense_decoder_block_gb300.stack import BeamSearch
    ddb, st = _stack(2, 64, 20)
    ids = workloads.make_token_ids(2, 20, VOCAB, seed=5).to(DEV).to(torch.int32)
    bs = BeamSearch(st, 4, 15)
    with pytest.raises(RuntimeError):
        bs.step()
    bs.begin(ids)
    with pytest.raises(RuntimeError):
        bs.begin(ids)
    for _ in range(14):
        bs.step()
    with pytest.raises(RuntimeError):
        bs.step()
    want = [t.clone() for t in bs.sequences()]
    bs.end()
    bs.begin(ids)
    bs.step()                                       # every kernel has run before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bs.step()
    for _ in range(13):
        graph.replay()
    got = bs.sequences()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bs.poll_error() == 0
    bs.end()
    assert bs.pool.tolist() == [bs.n_pages, 0]


def test_beam_search_refusals():
    from dense_decoder_block_gb300.stack import BeamSearch
    _, st = _stack(2, 64, 20)
    for args in (dict(beams=0, max_new=4), dict(beams=17, max_new=4), dict(beams=2, max_new=0), dict(beams=2, max_new=64)):
        with pytest.raises(ValueError):
            BeamSearch(st, **args)
    bs = BeamSearch(st, 2, 50)
    with pytest.raises(ValueError):
        bs.begin(torch.zeros(2, 20, dtype=torch.int32, device=DEV))


def test_beam_search_replayed_beyond_its_tokens():
    """Replays beyond max_new write no page that no beam was given, report an error and give no sequences; the
    next search is whole again."""
    from dense_decoder_block_gb300.stack import BeamSearch
    _, st = _stack(2, 64, 20)
    ids = workloads.make_token_ids(2, 20, VOCAB, seed=5).to(DEV).to(torch.int32)
    bs = BeamSearch(st, 4, 6)
    bs.begin(ids)
    for _ in range(5):
        bs.step()
    want = [t.clone() for t in bs.sequences()]
    bs.end()
    bs.begin(ids)
    bs.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bs.step()
    planned = set(bs.home[bs.home >= 0].tolist())
    rest = [p for p in range(bs.n_pages) if p not in planned]
    assert rest, "the pool has pages that no beam was given"
    before = [(c.k[rest].clone(), c.v[rest].clone()) for c in bs.caches.caches]
    for _ in range(20):                              # past the 6 tokens and the planned pages' 32 positions
        graph.replay()
    with pytest.raises(RuntimeError):
        bs.sequences()
    assert bs.poll_error() != 0
    for c, (k, v) in zip(bs.caches.caches, before):
        assert torch.equal(c.k[rest], k) and torch.equal(c.v[rest], v)
    while bs.poll_error():                           # one block's word after the other
        pass
    bs.end()
    assert bs.pool.tolist() == [bs.n_pages, 0]
    bs.begin(ids)
    for _ in range(5):
        bs.step()
    got = bs.sequences()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bs.poll_error() == 0


def test_beam_search_refuses_stacks_that_cannot_step():
    from types import SimpleNamespace

    from dense_decoder_block_gb300.stack import BeamSearch
    _, st = _stack(2, 64, 20)
    for heads, dtype, vocab in (((4, 2), torch.float32, VOCAB), ((12, 4), torch.bfloat16, VOCAB),
                                ((4, 2), torch.bfloat16, 2)):
        like = SimpleNamespace(dims=SimpleNamespace(n_heads=heads[0], n_kv_heads=heads[1]),
                               w_embed=torch.zeros(1, dtype=dtype, device=DEV), batch=2, max_seq=64, vocab=vocab,
                               blocks=st.blocks)
        with pytest.raises(ValueError):
            BeamSearch(like, 3, 4)


@pytest.mark.parametrize("shape,dtype", [((1, 20), torch.int32), ((2, 20), torch.int64), ((2, 0), torch.int32),
                                         ((2, 21), torch.int32), ((40,), torch.int32)])
def test_beam_search_refuses_prompts(shape, dtype):
    from dense_decoder_block_gb300.stack import BeamSearch
    _, st = _stack(2, 64, 20)
    bs = BeamSearch(st, 2, 4)
    with pytest.raises(ValueError):
        bs.begin(torch.zeros(shape, dtype=dtype, device=DEV))
    with pytest.raises(RuntimeError):
        bs.step()                                    # no search has begun
