"""BeamSearch.poll_error gives every code on record, one at a time."""
import pytest
import torch

from tests.test_gpu_beam_search import _stack

pytestmark = pytest.mark.gpu


def test_a_blocks_code_does_not_hide_the_searchs_own():
    import dense_decoder_block_gb300 as ddb
    from dense_decoder_block_gb300.stack import BeamSearch
    _, st = _stack(2, 64, 20)
    bs = BeamSearch(st, 2, 4)
    bs.err.fill_(ddb.LLAMA_ERR_NO_PAGES)
    st.blocks[0].selftest_wait_timeout(1_000_000)    # 1 ms
    torch.cuda.synchronize()
    assert bs.poll_error() == ddb.LLAMA_ERR_DEVICE_TIMEOUT
    assert bs.poll_error() == ddb.LLAMA_ERR_NO_PAGES
    assert bs.poll_error() == 0


def test_ids_out_of_range_are_reported():
    """In the prompt (the prefill's word) as in a step (the search's)."""
    import dense_decoder_block_gb300 as ddb
    from dense_decoder_block_gb300.stack import BeamSearch
    _, st = _stack(2, 64, 20)
    bs = BeamSearch(st, 2, 4)
    ids = torch.zeros(2, 20, dtype=torch.int32, device="cuda")
    ids[1, 3] = st.vocab
    bs.begin(ids)
    assert bs.poll_error() == ddb.LLAMA_ERR_INVALID_ARG and bs.poll_error() == 0
    bs.step()
    assert bs.poll_error() == 0
    bs.end()
    ids[1, 3] = 0
    bs.begin(ids)
    assert bs.poll_error() == 0
