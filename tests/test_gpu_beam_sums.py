"""The sums of exponentials in beam selection's long slices."""
import numpy as np
import pytest
import torch

from tests import paged_ref as ref
from tests.test_gpu_beam import _ddb, _select

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("offset", [0.0, 500.0])
def test_select_sums_of_long_slices(offset):
    """2^20 nearly equal logits, every 1024th the largest: the terms are 1 and t = e^-0.00099, whose sum in
    one fp32 chain of 512 loses 0.45 of a last place at each addition above 256, 104 units of 2^-24 in all.

    Here no maximum rises after a chunk's first logits, so of the scan's bound there remain 4 (ex2) + 15 + 31
    + 1 (additions) + 6 (the slices' join) + 1 (the distance's two roundings, 2.25 of 0.001, and the
    normaliser's 2^-36) = 58 units in the logarithm.  The logits' own rounding is no error: the reference
    takes the same ones.  Scores of about 0 leave the output's rounding out."""
    ddb = _ddb()
    d = -float(np.log((32735 + 0.45) * 2.0 ** -15))
    logits = torch.full((1, 1 << 20), offset - d)
    logits[0, ::1024] = offset
    scores = torch.tensor([13.862])
    got = _select(ddb, logits, scores, 1, 4)
    want = ref.beam_select(logits.double().numpy(), scores.double().numpy(), 1, 4)
    assert got[1].tolist() == [list(range(0, 4096, 1024))]
    assert np.all(np.abs(got[2] - want[2]) <= 58 * 2.0 ** -24 + 2.0 ** -24 * np.abs(want[2]))
