"""Rows that share pages beside the calls that know nothing of sharing: what stays on the stack's side of the contract."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
PS, N_PAGES, ROWS, COLUMNS = 16, 40, 6, 8


def _ddb():
    import dense_decoder_block_gb300 as ddb
    ddb.lib()
    return ddb


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("order", [(0, 1, 2), (2, 1, 0), (1, 0, 2)])
def test_rejected_drafts_are_released_and_shared_pages_given_up(order):
    """A prompt of 40 positions is forked twice; one row plans 30 drafted positions and releases the pages of the 25 that
    are rejected; then the rows are given up one by one while another request takes pages: shared pages stay off the stack,
    and keep their contents, until their last row is given up."""
    ddb = _ddb()
    gen = torch.Generator().manual_seed(1)
    k, v = (torch.randn(N_PAGES, 1, PS, 128, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2))
    caches = ddb.PagedCacheList([ddb.PagedCache(k, v)])
    free, pool = torch.randperm(N_PAGES, generator=gen).to(torch.int32).to(DEV), _i32([N_PAGES, 0])
    table, refs, err = _i32(np.full((ROWS, COLUMNS), -1)), _i32([0] * N_PAGES), _i32([0])
    ws = torch.empty(max(ddb.llama_paged_fork_workspace_bytes(2), ddb.llama_paged_free_workspace_bytes(1, N_PAGES)),
                     dtype=torch.uint8, device=DEV)

    def plan(row, start, count):
        slots = _i32(np.zeros((1, count)))
        ddb.llama_paged_plan(_i32([start]), _i32([count]), PS, N_PAGES, free, pool, table[row:row + 1], slots, err_dev=err)

    def on_stack():
        return set(free[:int(pool[0])].tolist())
    plan(0, 0, 40)
    ddb.llama_paged_fork(_i32([0, 0]), _i32([1, 2]), _i32([40, 40]), refs, free, pool, table, caches, ws, err_dev=err)
    shared = table[0, :2].tolist()
    assert table[1, :2].tolist() == shared and table[2, :2].tolist() == shared and refs[shared].tolist() == [2, 2]
    before = k[shared].clone()
    at_fork = (free.clone(), pool.clone())
    plan(1, 40, 30)                                        # pages 3 and 4 of the row
    assert int(pool[0]) == int(at_fork[1][0]) - 2
    ddb.llama_paged_release(_i32([45]), _i32([25]), PS, N_PAGES, free, pool, table[1:2], err_dev=err)
    assert pool.tolist() == at_fork[1].tolist() and torch.equal(free, at_fork[0])
    assert refs[shared].tolist() == [2, 2] and not on_stack() & set(shared)
    lens = [40, 45, 40]
    for n, row in enumerate(order):
        ddb.llama_paged_free(_i32([row]), _i32([lens[row]]), PS, N_PAGES, refs, free, pool, table, ws, err_dev=err)
        if n < 2:
            assert not on_stack() & set(shared) and refs[shared].tolist() == [1 - n, 1 - n]
            # another request takes pages, writes them, and goes
            plan(4, 0, 100)
            taken = table[4, :7].long()
            assert not set(taken.tolist()) & set(shared)
            k[taken] = 0
            ddb.llama_paged_release(_i32([0]), _i32([100]), PS, N_PAGES, free, pool, table[4:5], err_dev=err)
            assert torch.equal(k[shared], before)
    assert pool.tolist() == [N_PAGES, 0] and on_stack() == set(range(N_PAGES)) and not refs.any() and int(err) == 0
