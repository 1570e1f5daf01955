"""Log probabilities of many rows (a CTA of 4 warps each, segments chosen by one warp) that hold NaN, infinities or nothing."""
import pytest
import torch

from tests.test_gpu_logprobs import DEV, NEG, _ddb, check, logits, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [150, 700, 20000])
@pytest.mark.parametrize("n", [1, 5, 32])
def test_not_a_number_in_many_rows(vocab, n):
    """As for few rows: NaN log probabilities and entropy, and alternatives that are different tokens of the vocabulary; the
    rows between are what they are without them."""
    ddb = _ddb()
    rows = 1300
    z = logits(rows, vocab, 5)
    want = run(ddb, z, None, n)
    bad = {0: (17, float("nan")), 4: (vocab - 1, float("inf")), 600: (slice(None), float("nan")), 601: (slice(5, 7), float("inf")),
           1299: (slice(0, vocab, 2), float("nan"))}
    for r, (at, value) in bad.items():
        z[r, at] = value
    z[602], z[603, 1:] = NEG, NEG
    tokens = torch.randint(0, vocab, (rows,), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(torch.int32)
    tokens[603] = 0
    out = run(ddb, z, tokens, n)
    for r in bad:
        assert torch.isnan(out[0][r]) and torch.isnan(out[1][r]) and torch.isnan(out[3][r]).all(), r
        ids = out[2][r].tolist()
        assert len(set(ids)) == n and all(0 <= i < vocab for i in ids), r
    rest = [r for r in range(rows) if r not in (*bad, 602, 603)]
    for a, b in zip(out[1:], want[1:]):
        assert torch.equal(a[rest], b[rest])
    few = [1, 3, 5, 602, 603, 1298]
    check(z[few], tokens[few], [t[few] for t in out])
