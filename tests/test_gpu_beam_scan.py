"""Beam selection where a warp of the scan takes more than one slice."""
import numpy as np
import pytest
import torch

from tests import paged_ref as ref
from tests.test_gpu_beam import _ddb, _draw, _select

pytestmark = pytest.mark.gpu


def _warps():
    """Above the warps of the scan's grid: 3 blocks of 8 warps on an SM."""
    return torch.cuda.get_device_properties(0).multi_processor_count * 24


def _check(ddb, logits, scores, beams, n_out, last=None, eos=-1):
    """The reference's candidates, rank by rank.  A row's log sum is off by at most 2^-16, so beams whose
    candidates are closer than 2^-15 may change places (thousands of groups hold such pairs): the candidate
    at a rank is then one of the same exact score within 2^-15.  Order within a beam and places at -inf are
    exact."""
    got = _select(ddb, logits, scores, beams, n_out, last, eos)
    lg, sc, la = logits.double().numpy(), scores.double().numpy(), None if last is None else last.numpy()
    want = ref.beam_select(lg, sc, beams, n_out, la, eos)
    fin = np.isfinite(want[2])
    same = (got[0] == want[0]) & (got[1] == want[1])
    assert np.all(same[~fin]) and np.all(got[2][~fin] == -np.inf)
    assert np.all(np.abs(got[2][fin] - want[2][fin]) <= 2.0 ** -16 + 2.0 ** -24 * np.abs(want[2][fin]))
    for g, i in zip(*np.nonzero(~same)):
        row, v = int(got[0][g, i]), int(got[1][g, i])
        assert g * beams <= row < (g + 1) * beams and 0 <= v < lg.shape[1]
        ended = la is not None and la[row] == eos
        assert not ended or v == eos
        z = lg[row] - lg[row].max()
        exact = sc[row] if ended else z[v] - np.log(np.exp(z).sum()) + sc[row]
        assert abs(exact - want[2][g, i]) <= 2.0 ** -15, (g, i)
    place = got[0].astype(np.int64) * lg.shape[1] + got[1]
    assert all(len(set(p)) == n_out for p in place.tolist())


def _ended(rows, vocab, seed):
    """Last tokens and scores with ended beams and beams at -inf alone, in turn and in runs longer than a
    grid's step through the rows."""
    gen = torch.Generator().manual_seed(seed)
    eos = vocab // 2
    last = torch.randint(0, vocab - 1, (rows,), generator=gen).to(torch.int32)
    last[last == eos] = vocab - 1
    scores = -10.0 * torch.rand(rows, generator=gen)
    idle = torch.rand(rows, generator=gen)
    last[idle < 0.2] = eos
    scores[(idle > 0.4) & (idle < 0.5)] = float("-inf")
    q = rows // 8
    last[q:2 * q] = eos                       # a run of ended rows
    scores[3 * q:4 * q:2] = float("-inf")     # every other one at -inf
    scores[5 * q:6 * q] = float("-inf")       # a run at -inf
    last[rows - 3:] = eos                     # the last rows are not read
    return last, scores, eos


@pytest.mark.parametrize("vocab,n_out", [(1000, 4), (1003, 40), (3000, 4), (3001, 33), (64, 64)])
def test_select_with_more_rows_than_warps(vocab, n_out):
    """Rows behind the first grid's worth: stages, lists, bounds and sums of a warp's next slice, past rows
    that are not read."""
    ddb = _ddb()
    beams = 4
    groups = (_warps() + _warps() // 2) // beams + 3
    logits, scores = _draw(groups * beams, vocab, vocab)
    _check(ddb, logits, scores, beams, n_out)
    last, scores, eos = _ended(groups * beams, vocab, vocab + 1)
    _check(ddb, logits, scores, beams, n_out, last, eos)
    logits[::7, : vocab // 2] = float("-inf")
    _check(ddb, logits, scores, beams, n_out, last, eos)


@pytest.mark.parametrize("vocab,n_out", [(33000, 5), (32769, 64)])
def test_select_with_more_slices_than_warps(vocab, n_out):
    """Rows of two slices and more, so that a warp's slices lie in the middle of rows too."""
    ddb = _ddb()
    beams = 2
    groups = _warps() // 2 // beams + 40
    logits, _ = _draw(16, vocab, 3)
    logits = logits.repeat(groups * beams // 16 + 1, 1)[: groups * beams]
    last, scores, eos = _ended(groups * beams, vocab, 9)
    _check(ddb, logits, scores, beams, n_out, last, eos)


def test_select_rows_beyond_the_warps_equal_the_same_rows_alone():
    """A row's result does not depend on the rows that its warp took before it, bit for bit, where the
    slices are cut alike."""
    ddb = _ddb()
    vocab, n_out = 1000, 8
    rows = 2 * _warps() + 100
    logits, scores = _draw(rows, vocab, 4)
    whole = _select(ddb, logits, scores, 1, n_out)
    pick = torch.arange(rows - 1, 0, -97)
    alone = _select(ddb, logits[pick], scores[pick], 1, n_out)
    assert np.array_equal(whole[1][pick], alone[1]) and np.array_equal(whole[2][pick], alone[2])
    assert np.array_equal(whole[0][pick], np.repeat(pick.numpy()[:, None], n_out, 1))
