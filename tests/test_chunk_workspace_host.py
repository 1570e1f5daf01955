"""What the chunk attention asks for as a workspace (no GPU needed)."""
import pytest


@pytest.fixture(scope="module")
def need():
    from dense_decoder_block_gb300 import _native, build
    return _native.load(build.build()).llama_paged_chunk_attention_workspace_bytes


def test_sizes_that_the_call_refuses_need_none(need):
    assert need(65535, 1, 8, 2, 128, 64) > 0 and need(1, 2 ** 31 - 1, 8, 2, 128, 64) > 0
    for args in ((65536, 1, 8, 2, 128, 64), (65535, 32769, 8, 2, 128, 64), (2, 2 ** 30, 8, 2, 128, 64), (-1, 1, 8, 2, 128, 64),
                 (1, -1, 8, 2, 128, 64), (1, 1, 8, 2, 128, -1)):
        assert need(*args) == 0, args


@pytest.mark.gpu
def test_block_sizes_that_the_call_refuses_need_none():
    import torch

    import dense_decoder_block_gb300 as ddb
    import workloads
    dims = workloads.BlockDims(512, 8, 2, 128, 1024)
    w, g = workloads.make_weights(dims)
    dev = torch.device("cuda:0")
    blk = ddb.LlamaBlock(dims, {k: t.to(dev) for k, t in w.items()}, {k: t.to(dev) for k, t in g.items()}, 64)
    assert ddb.llama_block_prefill_paged_workspace_bytes(blk.h, 65535, 1) > 0
    assert ddb.llama_block_prefill_paged_workspace_bytes(blk.h, 1, 2 ** 30 - 1) > 0
    for batch, tokens in ((65536, 1), (65535, 16385), (1, 2 ** 30), (2, 2 ** 29), (0, 1), (1, 0), (-1, 1)):
        assert ddb.llama_block_prefill_paged_workspace_bytes(blk.h, batch, tokens) == 0, (batch, tokens)
