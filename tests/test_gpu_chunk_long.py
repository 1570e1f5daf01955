"""Chunk attention behind very long caches: what the sums over a row's keys lose must not grow with their number.  The table
names one page again and again, so that a cache of millions of positions takes one page."""
import numpy as np
import pytest
import torch

from tests.chunk_ref import U, ceil_div, chunk_tol

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
PS = 1024


def _ddb():
    import dense_decoder_block_gb300 as ddb
    ddb.lib()
    return ddb


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def attend(q, k, v, held):
    """q [T, Hq, D] behind `held` positions, all on one page of k, v [Hkv, PS, D]."""
    ddb = _ddb()
    T, Hq, D = q.shape
    L, Hkv = held + T, k.shape[0]
    table = torch.zeros(1, ceil_div(L, PS), dtype=torch.int32, device=DEV)
    o, err = torch.full_like(q, 7.0)[None], _i32([0])
    ws = torch.full((ddb.llama_paged_chunk_attention_workspace_bytes(1, T, Hq, Hkv, D, L),), 0xff, dtype=torch.uint8, device=DEV)
    ddb.llama_paged_chunk_attention(q[None].contiguous(), ddb.PagedCache(k[None].contiguous(), v[None].contiguous()), table, _i32([held]),
                                    _i32([T]), L, o, ws, err_dev=err)
    assert int(err) == 0
    return o[0]


def inputs(T, Hq, Hkv, D, dtype, scores, seed=1):
    """Random q and K (q = 0: equal scores), and one value per head and column, of magnitude 1 to 2, at every position."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randn(T, Hq, D, generator=gen, device=DEV).to(dtype)
    k = torch.randn(Hkv, PS, D, generator=gen, device=DEV).to(dtype)
    v = 1 + torch.rand(Hkv, 1, D, generator=gen, device=DEV)
    v = torch.where(torch.rand(v.shape, generator=gen, device=DEV) < 0.5, -v, v).to(dtype)
    return (q if scores == "random" else torch.zeros_like(q)), k, v.expand(Hkv, PS, D).contiguous(), v[:, 0].repeat_interleave(Hq // Hkv, 0)


# new tokens, query heads, KV heads: whole tiles of two halves; of one half, its chunks shared by two streams (152 KV heads
# would be needed for whole tiles: split); few rows split over all SMs
@pytest.mark.parametrize("scores", ["equal", "random"])
@pytest.mark.parametrize("T,Hq,Hkv,held", [(9728, 4, 1, 1 << 17), (9728, 4, 1, 1 << 20), (9728, 4, 1, 1 << 22), (9728, 4, 1, 1 << 24),
                                           (16, 32, 8, 1 << 22), (16, 4, 1, 1 << 24), (32, 608, 152, 300000)])
def test_rows_of_one_value_keep_it_bf16(T, Hq, Hkv, held, scores):
    """The sum of rounded weights times v, divided by their sum, is v up to the sums' own roundings.  Those of O are cut off
    (2^-23 each) at 8 additions a chunk of 128 keys, 512 chunks at most before they are carried over in fp32: 2^-11; carried
    over and joined: 3 roundings each, 2^24 / 2^16 + 152 times at most; those of l: 4 chains of 32 a chunk, 3 a chunk carried
    over.  Together below 2^-10, half of what separates v from the middle to the next bf16 (2^-9 |v|): the bits of v."""
    q, k, v, want = inputs(T, Hq, Hkv, 128, BF, scores)
    o = attend(q, k, v, held)
    off = int((o != want).sum())
    assert off == 0, f"{off} of {o.numel()}, {float((o.double() / want.double() - 1).abs().max()):.2e}"


@pytest.mark.parametrize("scores", ["equal", "random"])
@pytest.mark.parametrize("T,Hq,Hkv,D,held", [(4096, 4, 2, 64, 1 << 14), (4096, 4, 2, 64, 1 << 17), (2432, 8, 8, 128, 1 << 17),
                                             (4096, 4, 2, 32, 1 << 18), (64, 4, 2, 64, 1 << 20), (3, 8, 8, 128, 1 << 20)])
def test_rows_of_one_value_keep_it_fp32(T, Hq, Hkv, D, held, scores):
    """As above in fp32: 2048 products are added up one by one before they are carried over, sums over 64 keys in trees; each
    carrying over, and each joining of a piece, rounds three times.  O and l are off by that much each."""
    q, k, v, want = inputs(T, Hq, Hkv, D, F32, scores)
    o = attend(q, k, v, held)
    n = 2048 + 3 * ceil_div(held + T, 2048) + 3 * 304 + 16
    off = float((o.double() / want.double() - 1).abs().max())
    assert off <= 2 * n * U, f"{off:.2e}, bound {2 * n * U:.2e}"


@pytest.mark.parametrize("dtype,T,Hq,Hkv,D,held", [(BF, 9728, 4, 1, 128, (1 << 20) + 77), (BF, 40, 16, 2, 128, 3000001), (F32, 4096, 4, 2, 64, 100003),
                                                   (F32, 5, 4, 2, 32, 1000001)])
def test_random_values(dtype, T, Hq, Hkv, D, held):
    """Random values against the same sums in 64 bits, each key of the page counted as often as the row sees it; a late key
    that outweighs all before it for some rows (their sums so far are scaled down), an early one for others."""
    gen = torch.Generator(device=DEV).manual_seed(4)
    q = torch.randn(T, Hq, D, generator=gen, device=DEV).to(dtype)
    k, v = (torch.randn(Hkv, PS, D, generator=gen, device=DEV).to(dtype) for _ in range(2))
    o = attend(q, k, v, held).double()
    group = Hq // Hkv
    some = sorted({0, 1, T // 2, T - 1})
    for h in range(Hq):
        s = (q[some, h].double() @ k[h // group].double().T) * D ** -0.5
        reach = float(((q[some, h].double().abs() @ k[h // group].double().abs().T) * D ** -0.5).max())
        seen = torch.tensor(some, device=DEV)[:, None] + held + 1
        times = (seen - 1 - torch.arange(PS, device=DEV)[None]) // PS + 1
        w = torch.exp(s - s.amax(1, keepdim=True)) * times
        w /= w.sum(1, keepdim=True)
        vv = v[h // group].double()
        want, mass = w @ vv, w @ vv.abs()
        # the sums' share of that bound, 2 (3 L / 64 + 1052) 2^-24, at a length that covers what they lose at any: bf16 8192
        # (O, see above) + 3 * 46 + 3 * 304 in O and 600 + 3 * 46 + 3 * 304 in l, fp32 2048 + 3 * 49 + 3 * 304 in each
        tol = chunk_tol(want, mass, reach, dtype, D, 1 << 17 if dtype == BF else 1 << 16)
        assert float(((o[some, h] - want).abs() - tol).max()) <= 0, h


def test_infinities_where_a_piece_is_parted():
    """Whole tiles of 9728 tokens from position 60000 on: one of them ends its first 512 chunks among its own new positions.
    Infinities and NaN among the values there reach the rows that see them, in their columns alone, and no row before."""
    ddb = _ddb()
    T, held, D = 9728, 60000, 128
    gen = torch.Generator(device=DEV).manual_seed(6)
    q = torch.randn(1, T, 4, D, generator=gen, device=DEV).to(BF)
    pk, pv = (torch.randn(3, 1, PS, D, generator=gen, device=DEV).to(BF) for _ in range(2))
    table = torch.zeros(1, ceil_div(held + T, PS), dtype=torch.int32, device=DEV)
    table[0, 63], table[0, 64] = 1, 2                    # positions 64512 .. 66559 have pages of their own
    ws = torch.empty(ddb.llama_paged_chunk_attention_workspace_bytes(1, T, 4, 1, D, held + T), dtype=torch.uint8, device=DEV)
    outs = []
    for poison in (False, True):
        v = pv.clone()
        if poison:
            for pos, col, value in ((65510, 5, "inf"), (65540, 17, "nan"), (65550, 5, "-inf"), (65559, 40, "inf")):
                v[1 + (pos >= 65536), 0, pos % PS, col] = float(value)
        o, err = torch.full_like(q, 7.0), _i32([0])
        ddb.llama_paged_chunk_attention(q, ddb.PagedCache(pk, v), table, _i32([held]), _i32([T]), held + T, o, ws, err_dev=err)
        assert int(err) == 0
        outs.append(o[0])
    want, o = outs
    at = lambda pos: pos - held   # noqa: E731
    clean = [c for c in range(D) if c not in (5, 17, 40)]
    assert torch.equal(o[:, :, clean], want[:, :, clean]) and torch.isfinite(want.float()).all()
    for col, first in ((5, 65510), (17, 65540), (40, 65559)):
        assert torch.equal(o[:at(first), :, col], want[:at(first), :, col])
    assert torch.all(o[at(65510):at(65550), :, 5] == float("inf")) and torch.isnan(o[at(65550):, :, 5]).all()
    assert torch.isnan(o[at(65540):, :, 17]).all() and torch.all(o[at(65559):, :, 40] == float("inf"))
