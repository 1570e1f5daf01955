"""What BeamSearch refuses when it is made, so that no search stops in the middle."""
from types import SimpleNamespace

import pytest
import torch

import workloads
from tests.test_gpu_beam_search import DEV, _stack
from tests.test_gpu_stack import VOCAB

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("args", [dict(eos=VOCAB), dict(eos=2 ** 31 - 1), dict(page_size=0), dict(page_size=8),
                                  dict(page_size=24), dict(page_size=2048), dict(page_size=-16)],
                         ids=lambda a: "-".join(map(str, *a.items())))
def test_refused_when_made(args):
    from dense_decoder_block_gb300.stack import BeamSearch
    _, st = _stack(2, 64, 20)
    with pytest.raises(ValueError):
        BeamSearch(st, 2, 4, **args)


def test_stacks_that_the_calls_refuse():
    from dense_decoder_block_gb300.stack import BeamSearch
    _, st = _stack(1, 64, 20)

    def like(**other):
        return SimpleNamespace(**{**dict(dims=st.dims, w_embed=st.w_embed, batch=1, max_seq=64, vocab=VOCAB,
                                         blocks=st.blocks), **other})
    for other in (dict(blocks=st.blocks * 129), dict(vocab=(1 << 20) + 1), dict(max_seq=1 << 30)):
        with pytest.raises(ValueError):
            BeamSearch(like(**other), 2, 4)


@pytest.mark.parametrize("eos", [0, VOCAB - 1, -5])
def test_the_ends_of_the_vocabulary_may_end_beams(eos):
    from dense_decoder_block_gb300.stack import BeamSearch
    _, st = _stack(2, 64, 20)
    bs = BeamSearch(st, 2, 4, eos=eos, page_size=1024)
    bs.begin(workloads.make_token_ids(2, 20, VOCAB, seed=5).to(DEV).to(torch.int32))
    for _ in range(3):
        bs.step()
    tokens, scores = bs.sequences()
    assert tokens.shape == (2, 2, 4) and bool(torch.isfinite(scores).all()) and bs.poll_error() == 0
    bs.end()
