"""Log probabilities of given tokens, entropies and top alternatives against plain 64-bit forms."""
import numpy as np
import pytest
import torch

from tests import chunk_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NEG = float("-inf")


def _ddb():
    import dense_decoder_block_gb300 as ddb
    ddb.lib()
    return ddb


def run(ddb, z, tokens, n, err=None, stream=None):
    R = z.shape[0]
    out = [torch.full((R,), 9.0, device=DEV), torch.full((R,), 9.0, device=DEV),
           torch.full((R, n), -9, dtype=torch.int32, device=DEV), torch.full((R, n), 9.0, device=DEV)]
    ddb.llama_token_logprobs(z, tokens, None if tokens is None else out[0], entropy=out[1], top_ids=out[2] if n else None,
                             top_logprobs=out[3] if n else None, err_dev=err, stream=stream)
    return out


def check(z, tokens, out):
    V = z.shape[1]
    zs, (lp, h, ids, top) = z.cpu().numpy(), [t.cpu().numpy() for t in out]
    tokens = [None] * len(zs) if tokens is None else tokens.tolist()
    for r, token in enumerate(tokens):
        if token is not None and not 0 <= token < V:
            assert lp[r] == 9 and h[r] == 9 and (ids[r] == -9).all() and (top[r] == 9).all()
            continue
        want = ref.token_logprobs(zs[r], token, ids.shape[1])
        assert np.array_equal(ids[r], want[2]), f"row {r}"
        finite = np.isfinite(want[3])
        assert np.array_equal(top[r][~finite], want[3][~finite])
        zf = zs[r].astype(np.float64)
        x = zf[want[2]][finite]
        bound = [ref.logprob_tol(a, np.array([b, zf.max()]), V)[0] for a, b in zip(want[3][finite], x)]
        assert (np.abs(top[r][finite] - want[3][finite]) <= bound).all(), f"row {r}"
        assert abs(h[r] - want[1]) <= ref.entropy_tol(want[1], V), f"row {r}: {h[r]} {want[1]}"
        if token is not None:
            if np.isinf(want[0]):
                assert lp[r] == want[0]
            else:
                assert abs(lp[r] - want[0]) <= ref.logprob_tol(want[0], np.array([zf[token], zf.max()]), V)[0], f"row {r}"


def logits(rows, vocab, seed, scale=3.0):
    return torch.randn(rows, vocab, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV) * scale


@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 127, 128, 511, 513, 1000, 4099, 32000, 128256, 1 << 20])
@pytest.mark.parametrize("rows", [1, 2, 33])
def test_matches_reference(rows, vocab):
    ddb = _ddb()
    z = logits(rows, vocab, vocab)
    tokens = torch.randint(0, vocab, (rows,), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(torch.int32)
    tokens[0] = z[0].argmax()
    for n in sorted({0, 1, min(5, vocab), min(32, vocab)}):
        check(z, tokens, run(ddb, z, tokens, n))


@pytest.mark.parametrize("rows", [5, 151, 152, 153, 400, 1300])
def test_many_rows_and_skipped_ones(rows):
    ddb = _ddb()
    z = logits(rows, 2051, rows)
    tokens = torch.randint(0, 2051, (rows,), device=DEV, generator=torch.Generator(device=DEV).manual_seed(2)).to(torch.int32)
    tokens[::3] = -1
    z[::3] = float("nan")                    # not read
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    check(z, tokens, run(ddb, z, tokens, 7, err))
    assert int(err) == 0
    tokens[1], tokens[rows - 1] = 2051, 2 ** 31 - 1
    check(z, tokens, run(ddb, z, tokens, 7, err))
    assert int(err) == -1


def test_without_tokens_and_entropy():
    ddb = _ddb()
    z = logits(3, 1003, 3)
    full = run(ddb, z, torch.zeros(3, dtype=torch.int32, device=DEV), 4)
    out = run(ddb, z, None, 4)
    assert torch.equal(out[1], full[1]) and torch.equal(out[2], full[2]) and torch.equal(out[3], full[3])
    lp = torch.zeros(3, device=DEV)
    ddb.llama_token_logprobs(z, torch.zeros(3, dtype=torch.int32, device=DEV), lp)
    assert torch.equal(lp, full[0])


@pytest.mark.parametrize("vocab", [50, 3001, 128256])
def test_masks_ties_and_wide_rows(vocab):
    """-inf, the type's lowest value, equal logits (the lowest token first), signed zeros, one logit above all, ascending
    and descending rows, rows whose mask leaves one logit or none."""
    ddb = _ddb()
    z = logits(14, vocab, 4)
    low = torch.finfo(torch.float32).min
    z[0, 1::2] = NEG
    z[1, : vocab - 1] = NEG
    z[2] = NEG
    z[3] = low
    z[4, 3:] = low
    z[5] = 0.25
    z[6] = 0.0
    z[6, ::2] = -0.0
    z[7] = torch.arange(vocab, device=DEV) * 1e-3
    z[8] = -torch.arange(vocab, device=DEV) * 1e-3
    z[9, vocab // 2] = 200.0
    z[10] = (z[10] * 2).round() / 2
    z[11] = torch.arange(vocab, device=DEV) // 7 * 0.5
    z[12] *= 1e4
    z[13, 0], z[13, vocab - 1] = 60.0, 60.0
    tokens = torch.randint(0, vocab, (14,), device=DEV, generator=torch.Generator(device=DEV).manual_seed(3)).to(torch.int32)
    tokens[1], tokens[9] = vocab - 1, vocab // 2
    for n in (1, 5, 32):
        check(z, tokens, run(ddb, z, tokens, n))


@pytest.mark.parametrize("rows", [14, 1300])
@pytest.mark.parametrize("vocab", [161, 250, 257, 512, 513, 700, 1290, 4584, 16390])
def test_rows_of_few_segments(rows, vocab):
    """Vocabularies with fewer segments than alternatives, and rows in order or of few values, in both ways of sharing rows
    out; equal logits everywhere, too."""
    ddb = _ddb()
    z = logits(rows, vocab, 8)
    z[1] = torch.arange(vocab, device=DEV) * 1e-3
    z[2] = -torch.arange(vocab, device=DEV) * 1e-3
    z[3] = (z[3] * 2).round() / 2
    z[4] = 0.25
    z[5] = NEG
    z[6, 3:] = NEG
    z[7, : vocab // 2] = torch.finfo(torch.float32).min
    z[8, vocab - 1] = 50.0
    z[9, ::2] = 3.0
    tokens = torch.randint(0, vocab, (rows,), device=DEV, generator=torch.Generator(device=DEV).manual_seed(3)).to(torch.int32)
    for n in (1, 2, 7, 20, 32):
        out = run(ddb, z, tokens, n)
        check(z[:14], tokens[:14], [t[:14] for t in out])


def test_peaked_rows_keep_small_probabilities():
    """A top logit far above the rest: its log probability and the entropy are small, and not rounded to zero."""
    ddb = _ddb()
    z = torch.zeros(6, 5000, device=DEV)
    for r, gap in enumerate((10.0, 15.0, 20.0, 25.0, 30.0, 40.0)):
        z[r, 1234] = gap
    tokens = torch.full((6,), 1234, dtype=torch.int32, device=DEV)
    out = run(ddb, z, tokens, 2)
    for r in range(6):
        lp, h, ids, top = ref.token_logprobs(z[r].cpu().numpy(), 1234, 2)
        d = np.exp(-float(z[r, 1234])) * 4999
        want = -np.log1p(d)
        assert abs(float(out[0][r]) - want) <= 400 * ref.U * abs(want)
        want_h = np.log1p(d) + d * float(z[r, 1234]) / (1 + d)
        assert abs(float(out[1][r]) - want_h) <= 400 * ref.U * want_h
        assert out[2][r].tolist() == ids.tolist()


@pytest.mark.parametrize("vocab", [700, 128256])
def test_not_a_number(vocab):
    ddb = _ddb()
    z = logits(5, vocab, 5)
    z[0, 17] = float("nan")
    z[1, vocab - 1] = float("inf")
    z[2] = float("nan")
    z[3, 5] = float("inf")
    z[3, 6] = float("inf")
    tokens = torch.tensor([17, 3, 4, 5, 6], dtype=torch.int32, device=DEV)
    out = run(ddb, z, tokens, 32)
    assert torch.isnan(out[0][:4]).all() and torch.isnan(out[1][:4]).all() and torch.isnan(out[3][:4]).all()
    ids = out[2].long()
    assert bool(((ids >= 0) & (ids < vocab)).all())
    assert all(len(set(row.tolist())) == 32 for row in ids)
    check(z[4:], tokens[4:], [t[4:] for t in out])


def test_rows_off_16_bytes():
    """A vocabulary that is no multiple of 4, and logits that start off a 16-byte boundary."""
    ddb = _ddb()
    for off in (1, 2, 3):
        for vocab in (1021, 1022, 1024, 9):
            buf = logits(1, 6 * vocab + 8, 7 + off)[0]
            z = buf[off:off + 6 * vocab].view(6, vocab)
            tokens = torch.arange(6, dtype=torch.int32, device=DEV)
            check(z, tokens, run(ddb, z, tokens, min(9, vocab)))


def test_graph_and_stream():
    ddb = _ddb()
    z = logits(40, 5003, 8)
    tokens = torch.arange(40, dtype=torch.int32, device=DEV)
    want = run(ddb, z, tokens, 6)
    out = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ddb.llama_token_logprobs(z, tokens, out[0], out[1], out[2], out[3])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    z.copy_(logits(40, 5003, 9))
    graph.replay()
    torch.cuda.synchronize()
    check(z, tokens, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(ddb, z, tokens, 6)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, got))


def test_offsets_beyond_32_bits():
    ddb = _ddb()
    rows, vocab = 2100, 1 << 20
    z = torch.zeros(rows, vocab, device=DEV)
    assert z.numel() > 2 ** 31
    z[rows - 1] = logits(1, vocab, 11)[0]
    tokens = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    tokens[rows - 1] = 77
    out = run(ddb, z, tokens, 3)
    check(z[rows - 1:], tokens[rows - 1:], [t[rows - 1:] for t in out])
    assert torch.all(out[0][:-1] == 9)
