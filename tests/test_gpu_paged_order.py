"""A call of paged attention reads nothing before the kernels that the stream holds in front of it are done,
those among them that start their dependents early (the row-wise kernels) included."""
import pytest
import torch

from tests.test_gpu_paged import DEV, SHAPES, _ddb, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", ["8b", "mqa8", "group3", "group16", "f32-128"])
@pytest.mark.parametrize("ps", [16, 128])
def test_rows_written_by_the_kernel_in_front(shape, ps):
    """llama_rmsnorm writes every row of the pages (normalised keys, values), the attention follows at once:
    the result is the one that it gives after a wait."""
    ddb = _ddb()
    dtype, Hq, Hkv, D = SHAPES[shape]
    lens = [3000, 1, 2500, 0, 700]
    columns = -(-max(lens) // ps)
    n_pages = len(lens) * columns
    gen = torch.Generator().manual_seed(4)
    table = torch.randperm(n_pages, generator=gen).view(len(lens), columns).to(torch.int32).to(DEV)
    raw = [torch.randn(n_pages, Hkv, ps, D, generator=gen).to(dtype).to(DEV) for _ in range(2)]
    gain = (torch.rand(D, generator=gen) + 0.5).to(dtype).to(DEV)
    q = torch.randn(len(lens), Hq, D, generator=gen).to(dtype).to(DEV)
    kv = ddb.PagedCache(torch.empty_like(raw[0]), torch.empty_like(raw[0]))
    rows = n_pages * Hkv * ps
    ws = torch.empty(ddb.llama_paged_attention_workspace_bytes(len(lens), Hq, Hkv, D, 3000), dtype=torch.uint8, device=DEV)
    ln = _i32(lens)

    def norm():
        for x, y in zip(raw, (kv.k, kv.v)):
            ddb.llama_rmsnorm(x, gain, y, rows, D, 1e-5)

    def attend(o):
        ddb.llama_paged_attention(q, kv, table, ln, 3000, o, ws)
        return o

    norm()
    torch.cuda.synchronize()
    want = attend(torch.empty_like(q))
    torch.cuda.synchronize()
    assert bool(torch.isfinite(want).all())
    for _ in range(10):
        kv.k.fill_(float("nan"))
        kv.v.fill_(float("nan"))
        norm()
        got = attend(torch.empty_like(q))
        torch.cuda.synchronize()
        assert torch.equal(got, want)
