"""A step at a position out of range leaves nothing running that the next call on the stream could meet."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["devpos", "seqpos"])
@pytest.mark.parametrize("bad", [-1, 320])
def test_a_good_step_behind_a_bad_one(kind, bad):
    """The same workspace, no wait in between: the good step's bits are those that it gives alone, and the cache
    holds what it held."""
    import dense_decoder_block_gb300 as ddb
    dims, B, max_seq, P = workloads.BlockDims(1024, 8, 2, 128, 4096), 8, 320, 300
    dev = torch.device("cuda:0")
    w, g = workloads.make_weights(dims, weight_std=0.03)
    blk = ddb.LlamaBlock(dims, {k: t.to(dev) for k, t in w.items()}, {k: t.to(dev) for k, t in g.items()}, max_seq)
    kv = ddb.KVCache(*(t.to(dev) for t in workloads.make_cache(dims, B, max_seq, P, 1)))
    x, other = (workloads.make_x(B, 1, dims.d_model, seed=s).to(dev) for s in (3, 4))
    ws, n = blk.workspace(B, 1), 1 if kind == "devpos" else B
    good = torch.full((n,), P, dtype=torch.int32, device=dev)
    wrong = good.clone()
    wrong[-1] = bad

    def step(inp, pos):
        y = torch.empty_like(inp)
        (blk.decode_devpos if kind == "devpos" else blk.decode_seqpos)(inp, kv, pos, y, ws)
        return y

    want = step(x, good)
    torch.cuda.synchronize()
    assert blk.poll_error() == 0
    k, v = kv.k.clone(), kv.v.clone()
    got = []
    for _ in range(10):
        step(other, wrong)
        got.append(step(x, good))
    assert blk.poll_error() == ddb.LLAMA_ERR_POS_RANGE and blk.poll_error() == 0
    assert all(torch.equal(y, want) for y in got)
    bits = torch.int16                               # (rows behind the positions are NaN)
    assert torch.equal(kv.k.view(bits), k.view(bits)) and torch.equal(kv.v.view(bits), v.view(bits))
