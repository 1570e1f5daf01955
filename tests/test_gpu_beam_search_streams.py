"""Beam search whose buffers are filled on one stream and whose calls go to another."""
import pytest
import torch

import workloads
from tests.test_gpu_beam_search import DEV, _stack
from tests.test_gpu_stack import VOCAB

pytestmark = pytest.mark.gpu

BUSY = 20_000_000      # clock cycles that a stream is kept busy for: about 10 ms


def _ids(seed):
    ids = workloads.make_token_ids(2, 20, VOCAB, seed=seed).to(DEV).to(torch.int32)
    torch.cuda.synchronize()
    return ids


def _slow_fills(monkeypatch):
    """Fills of zeros that the stream reaches late."""
    zeros = torch.zeros

    def slow(*a, **k):
        torch.cuda._sleep(BUSY)
        return zeros(*a, **k)
    monkeypatch.setattr(torch, "zeros", slow)


def test_a_search_on_a_side_stream(monkeypatch):
    """Made on the current stream, with fills that are slow to come; begun, stepped and ended on a side stream."""
    from dense_decoder_block_gb300.stack import BeamSearch
    _, st = _stack(2, 64, 20)
    ids, side, got = _ids(5), torch.cuda.Stream(), []
    for stream in (None, side):
        with monkeypatch.context() as m:
            if stream is not None:
                _slow_fills(m)
            bs = BeamSearch(st, 4, 10, eos=3)
            assert torch.cuda.current_stream().query(), "fills are still to come"
        bs.begin(ids, stream)
        for _ in range(9):
            bs.step(stream)
        got.append(bs.sequences())
        assert bs.poll_error() == 0
        bs.end(stream)
    side.synchronize()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert bs.pool.tolist() == [bs.n_pages, 0] and bs.free.tolist() == list(range(bs.n_pages))


def test_results_are_read_before_the_next_calls(monkeypatch):
    """sequences() and poll_error() leave nothing on the current stream that a call on another one could
    overtake."""
    from dense_decoder_block_gb300.stack import BeamSearch
    _, st = _stack(2, 64, 20)
    ids, side = _ids(6), torch.cuda.Stream()
    bs = BeamSearch(st, 4, 10)
    bs.begin(ids, side)
    bs.step(side)
    want = [t.clone() for t in bs.sequences()]
    clone, zero = torch.Tensor.clone, torch.Tensor.zero_

    def late(f):
        def call(*a, **k):
            torch.cuda._sleep(BUSY)
            return f(*a, **k)
        return call
    with monkeypatch.context() as m:
        m.setattr(torch.Tensor, "clone", late(clone))
        m.setattr(torch.Tensor, "zero_", late(zero))
        got = bs.sequences()
        assert torch.cuda.current_stream().query(), "scores are still to be read"
        bs.err.fill_(-1)
        assert bs.poll_error() == -1
        assert torch.cuda.current_stream().query(), "the code is still to be cleared"
    bs.step(side)
    bs.end(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and bs.poll_error() == 0
