"""A stack whose buffers are filled on one stream and whose calls go to another."""
import pytest
import torch

import workloads
from tests.test_gpu_beam_search import DEV, _stack
from tests.test_gpu_stack import VOCAB

pytestmark = pytest.mark.gpu


def test_a_stack_made_on_another_stream(monkeypatch):
    """Fills that the current stream reaches late are done when the stack is made; prefill and steps on a side
    stream choose what they choose on the current one."""
    ids = workloads.make_token_ids(2, 20, VOCAB, seed=5).to(DEV).to(torch.int32)
    torch.cuda.synchronize()
    zeros, side, got, stacks = torch.zeros, torch.cuda.Stream(), [], []

    def slow(*a, **k):
        torch.cuda._sleep(20_000_000)                # about 10 ms
        return zeros(*a, **k)
    for stream in (None, side):
        with monkeypatch.context() as m:
            if stream is not None:
                m.setattr(torch, "zeros", slow)
            st = _stack(2, 64, 20)[1]
            stacks.append(st)                        # (one that is freed waits for the device)
            assert torch.cuda.current_stream().query(), "fills are still to come"
        st.prefill(ids, stream)
        for _ in range(3):
            st.decode_step(stream)
        torch.cuda.synchronize()
        assert st.poll_error() == 0
        got.append((st.ids.clone(), st.logits.clone(), int(st.pos)))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]) and got[0][2] == got[1][2] == 23
