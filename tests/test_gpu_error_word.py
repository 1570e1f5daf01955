"""The device error word: which of two errors it keeps."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu


def _block():
    import dense_decoder_block_gb300 as ddb
    dims = workloads.BlockDims(512, 8, 2, 128, 1024)
    w, g = workloads.make_weights(dims)
    dev = torch.device("cuda:0")
    blk = ddb.LlamaBlock(dims, {k: t.to(dev) for k, t in w.items()}, {k: t.to(dev) for k, t in g.items()}, 64)
    x = workloads.make_x(2, 1, 512).to(dev)
    pk = torch.zeros(8, 2, 16, 128, dtype=torch.bfloat16, device=dev)
    kv = ddb.PagedCache(pk, pk.clone())
    table = torch.arange(8, dtype=torch.int32, device=dev).view(2, 4)

    def step(pos, pages=table):
        blk.decode_paged(x, kv, pages, torch.tensor(pos, dtype=torch.int32, device=dev), torch.empty_like(x),
                         blk.workspace(2, 1))
        torch.cuda.synchronize()

    return ddb, blk, step, table


def test_an_expired_wait_replaces_another_error():
    """A paged step leaves a bad position or page on record and its other rows are good; a wait that expires
    after that leaves every row undefined, so its code is the one that the host reads."""
    ddb, blk, step, table = _block()
    bad = table.clone()
    bad[1, 1] = 8
    for pos, pages, code in (([64, 3], table, ddb.LLAMA_ERR_POS_RANGE), ([3, 16], bad, ddb.LLAMA_ERR_INVALID_ARG)):
        step(pos, pages)
        assert blk.poll_error() == code
        step(pos, pages)
        blk.selftest_wait_timeout(20_000_000)   # 20 ms
        assert blk.poll_error() == ddb.LLAMA_ERR_DEVICE_TIMEOUT
        assert blk.poll_error() == 0            # one word, read once


def test_an_expired_wait_is_not_replaced():
    ddb, blk, step, _ = _block()
    blk.selftest_wait_timeout(20_000_000)
    step([64, 3])
    assert blk.poll_error() == ddb.LLAMA_ERR_DEVICE_TIMEOUT
    step([5, 3])
    assert blk.poll_error() == 0
