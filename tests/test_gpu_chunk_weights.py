"""The weights of the bf16 chunk attention are rounded before their product with V, and the normaliser sums the rounded ones:
their roundings leave a row's output where it is when its keys hold like values."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16


def _ddb():
    import dense_decoder_block_gb300 as ddb
    ddb.lib()
    return ddb


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


# new tokens, positions in front of them, query heads, KV heads: both halves of a tile, one half whose chunks two streams
# share, tiles in rounds, tiles split over CTAs (the heavy keys in one piece or in several)
CALLS = {"pair": (100, 300, 8, 2), "streams": (4, 300, 8, 2), "rounds": (600, 700, 32, 8), "split": (20, 9000, 4, 1),
         "split-pair": (150, 6000, 4, 2), "group3": (50, 700, 6, 2)}


@pytest.mark.parametrize("call", CALLS)
def test_rows_of_one_value_keep_it(call):
    """Scores (log2) of row r: a = 1.02 q_r at a key of the first chunk, 1.5 a at a later key, -7 a at all others, q_r of 4 to
    8: the later key's weight lies 2^2 to 2^4 above that of the row's reference so far, and is rounded there.  Both keys
    hold the value v, and the others weigh 2^-34 of the later one at most: the exact row is v up to 9020 * 2^-34 * 3 |v|
    (|v| >= 1, |v'| <= 2), below 2^-19 |v|.  With p~ the rounded weights, O / l = sum p~ v / sum p~ is v up to the roundings
    of fp32 sums (2^-13 at most: the 1000 of the call's other bound, twice for sums that are cut off), and the middle
    between v and the next bf16 is 2^-9 |v| away at least: every element has the bits of v.  (A normaliser of weights that
    are not rounded is off by up to 2^-8, beyond the middle for many v.)"""
    ddb = _ddb()
    T, held, Hq, Hkv = CALLS[call]
    L, D, ps = held + T, 128, 16
    gen = torch.Generator(device=DEV).manual_seed(31)
    n = -(-L // ps)

    def signed(*shape):   # magnitudes of 1 to 2
        x = 1 + torch.rand(*shape, generator=gen, device=DEV)
        return torch.where(torch.rand(*shape, generator=gen, device=DEV) < 0.5, -x, x).to(BF)
    k = torch.zeros(Hkv, n * ps, D, dtype=BF, device=DEV)
    k[:, :, 0] = -56.0
    v = signed(Hkv, n * ps, D)
    for g in range(Hkv):
        early, late = 17 + g, held - 30 - 70 * g
        k[g, early, 0], k[g, late, 0] = 8.0, 12.0
        v[g, late] = v[g, early]
    q = torch.zeros(1, T, Hq, D, dtype=BF, device=DEV)
    q[..., 0] = (4 + 4 * torch.rand(1, T, Hq, generator=gen, device=DEV)).to(BF)
    table = torch.randperm(n, generator=gen, device=DEV)
    pk, pv = (torch.empty(n, Hkv, ps, D, dtype=BF, device=DEV) for _ in range(2))
    for pages, rows in ((pk, k), (pv, v)):
        pages[table] = rows.view(Hkv, n, ps, D).transpose(0, 1)
    o = torch.zeros_like(q)
    ws = torch.empty(ddb.llama_paged_chunk_attention_workspace_bytes(1, T, Hq, Hkv, D, L), dtype=torch.uint8, device=DEV)
    err = _i32([0])
    ddb.llama_paged_chunk_attention(q, ddb.PagedCache(pk, pv), table.to(torch.int32)[None].contiguous(), _i32([held]), _i32([T]),
                                    L, o, ws, err_dev=err)
    assert int(err) == 0
    for h in range(Hq):
        g = h // (Hq // Hkv)
        off = (o[0, :, h] != v[g, 17 + g]).sum()
        assert int(off) == 0, f"head {h}: {int(off)} of {T * D} elements"
