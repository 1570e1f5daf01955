"""The page pool's two words: the free count follows every plan and release, whatever the second word
held before."""
import numpy as np
import pytest
import torch

from tests import paged_ref as ref
from tests.test_gpu_paged import PLANS, _ddb, _i32, _plan_state, _same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("word", [7, -1, 1, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("out", [False, True], ids=["in-place", "pool-out"])
@pytest.mark.parametrize("name", ["step", "ragged", "wide", "many"])       # one block, and several
def test_second_word_holds_anything(name, out, word):
    ddb = _ddb()
    start, count, tokens, ps = PLANS[name]
    columns = max(ref.ceil_div(s + c, ps) for s, c in zip(start, count)) + 1
    n_pages, table, free, n_free = _plan_state(start, count, tokens, ps, columns, 3, 1)
    want = ref.plan(start, count, tokens, ps, n_pages, free, n_free, table)
    t, f, p, err = _i32(table), _i32(free), _i32([n_free, word]), _i32([0])
    q = _i32([-5, word]) if out else p
    slots = torch.full((len(start), tokens), -9, dtype=torch.int32, device="cuda")
    ddb.llama_paged_plan(_i32(start), _i32(count), ps, n_pages, f, p, t, slots, pool_out=q, err_dev=err)
    assert q.tolist() == [want[3], 0]
    _same((t.cpu().numpy(), slots.cpu().numpy(), f.cpu().numpy(), int(q[0]), int(err[0])), want)
    if out:
        assert p.tolist() == [n_free, word]
    # the pages that a second plan takes are others than the first one's
    q[1] = word
    again = torch.full_like(t, -1)
    few = _i32([0] * len(start)), _i32([0] * (len(start) - 1) + [min(tokens, ps)])
    ddb.llama_paged_plan(*few, ps, n_pages, f, q, again, slots, err_dev=err)
    taken = [int(x) for x in again.flatten() if x >= 0]
    assert q.tolist() == [want[3] - 1, 0] and len(taken) == 1 and taken[0] not in set(want[0].flatten().tolist())
    # and back
    q[1] = word
    ddb.llama_paged_release(*few, ps, n_pages, f, q, again, err_dev=err)
    back = _i32([0, word]) if out else q
    q[1] = word
    ddb.llama_paged_release(_i32(start), _i32(count), ps, n_pages, f, q, t, pool_out=back, err_dev=err)
    assert back.tolist() == [n_free, 0] and int(err[0]) == 0 and np.array_equal(f.cpu().numpy(), free)


def test_counts_in_place_with_refused_requests():
    """Several blocks in place: requests out of range are left out of the count, too few pages change nothing."""
    ddb = _ddb()
    B, ps, columns, tokens = 300, 16, 4, 20
    start, count = [0] * B, [(7 * i) % 21 for i in range(B)]
    start[5], count[9], start[200] = -1, 21, 60
    n_pages, table, free, n_free = _plan_state([0] * B, count, tokens, ps, columns, 0, 2)
    for have in (n_free, 10):
        want = ref.plan(start, count, tokens, ps, n_pages, free, have, table)
        t, f, p, err = _i32(table), _i32(free), _i32([have, 3]), _i32([0])
        slots = torch.full((B, tokens), -9, dtype=torch.int32, device="cuda")
        ddb.llama_paged_plan(_i32(start), _i32(count), ps, n_pages, f, p, t, slots, err_dev=err)
        assert p.tolist() == [want[3], 0] and np.array_equal(slots.cpu().numpy(), want[1])
        assert int(err[0]) in (-3, -7) if have == 10 else int(err[0]) == want[4] == -3
