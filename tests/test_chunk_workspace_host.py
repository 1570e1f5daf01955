"""What the chunk attention asks for as a workspace (no GPU needed)."""
import pytest


@pytest.fixture(scope="module")
def need():
    from dense_decoder_block_gb300 import _native, build
    return _native.load(build.build()).llama_paged_chunk_attention_workspace_bytes


def test_sizes_that_the_call_refuses_need_none(need):
    assert need(65535, 1, 8, 2, 128, 64) > 0 and need(1, 2 ** 31 - 1, 8, 2, 128, 64) > 0
    for args in ((65536, 1, 8, 2, 128, 64), (65535, 32769, 8, 2, 128, 64), (2, 2 ** 30, 8, 2, 128, 64), (-1, 1, 8, 2, 128, 64),
                 (1, -1, 8, 2, 128, 64), (1, 1, 8, 2, 128, -1)):
        assert need(*args) == 0, args


@pytest.mark.gpu
def test_block_sizes_that_the_call_refuses_need_none():
    import torch

    import dense_decoder_block_gb300 as ddb
    import workloads
    dims = workloads.BlockDims(512, 8, 2, 128, 1024)
    w, g = workloads.make_weights(dims)
    dev = torch.device("cuda:0")
    blk = ddb.LlamaBlock(dims, {k: t.to(dev) for k, t in w.items()}, {k: t.to(dev) for k, t in g.items()}, 64)
    assert ddb.llama_block_prefill_paged_workspace_bytes(blk.h, 65535, 1) > 0
    assert ddb.llama_block_prefill_paged_workspace_bytes(blk.h, 1, 2 ** 30 - 1) > 0
    for batch, tokens in ((65536, 1), (65535, 16385), (1, 2 ** 30), (2, 2 ** 29), (0, 1), (1, 0), (-1, 1)):
        assert ddb.llama_block_prefill_paged_workspace_bytes(blk.h, batch, tokens) == 0, (batch, tokens)


def _split(start, count, kv_heads, tq, ctas, seqs, join_keys, stretch, pieces):
    """CTAs that the tiles of a call's launches are split over (0: dealt out whole), by the rule of the kernels: tiles of tq
    tokens, each with the keys that its last token attends and 128 more."""
    most = 0
    for b in range(0, len(start), seqs):
        tiles = total = 0
        for s, c in zip(start[b:b + seqs], count[b:b + seqs]):
            for y in range(-(-c // tq)):
                tiles += kv_heads
                total += kv_heads * (s + min((y + 1) * tq, c) + 128)
        rounds = 1 + sum(tiles > i * ctas for i in (1, 2, 3))
        if tiles == 0 or tiles >= 4 * ctas or rounds * total <= (total / ctas + join_keys) * tiles:
            continue
        cap = min(total / stretch, pieces * (total * tiles / 128) ** 0.5)
        most = max(most, min(ctas, max(tiles, int(cap))))
    return most


def test_holds_the_pieces_of_every_split(need):
    """Two partials (m, l, o) of a tile's rows for each CTA that takes part, in both types, and 20 bytes for every CTA, for
    random calls and for those whose sequences are all as long as can be.  (A tile of fewer than four 128-key chunks is
    never cut.)"""
    import random
    rng = random.Random(5)

    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))
    split = 0
    for case in range(3000):
        kv, group = rng.choice([1, 2, 8]), rng.choice([1, 3, 4, 8, 64])
        batch, tokens = log(1, 1500), log(1, 600)
        most = tokens + log(1, 100000)
        full = case % 2
        count = [tokens if full else rng.choice([0, 1, rng.randint(0, tokens)]) for _ in range(batch)]
        start = [most - c if full else rng.randint(0, most - c) for c in count]
        for dim, tq, rows, ctas, rest in ((128, 2 * (128 // group), 256, 152, (1024, 768, 512, 2)),
                                          (128, 64 // group, 64, 152, (256, 64, 256, 4)), (64, 64 // group, 64, 304, (256, 64, 256, 4))):
            if batch * tokens > 20000:
                continue
            n = _split(start, count, kv, tq, ctas, *rest) if most >= 385 else 0    # fewer positions: no tile of 4 chunks
            split += n > 0
            assert need(batch, tokens, kv * group, kv, dim, most) >= 2 * n * rows * (dim + 2) * 4 + 304 * 20
    assert split > 500, split


def test_grows_with_the_call(need):
    """Small calls ask for little, larger ones for no less, and none for more than all CTAs' partials."""
    assert need(1, 1, 1, 1, 128, 384) == 304 * 20
    assert need(1, 1, 1, 1, 128, 385) < 1 << 20 and need(1, 16, 4, 2, 64, 1000) < 1 << 20
    # (CTAs, rows) of the type, and the keys from which on a row's O is carried over, in fp32 a row each
    for dim, ctas, rows, keys in ((128, 152, 256, 65536), (64, 304, 64, 2048), (32, 304, 64, 2048)):
        pieces, carried = 2 * ctas * rows * (dim + 2) * 4 + 304 * 20, ctas * rows * dim * 4
        assert need(8, 512, 32, 8, dim, keys) == pieces and need(8, 512, 32, 8, dim, keys + 1) == pieces + carried
        top = need(65535, 32768, 64, 8, dim, 2 ** 31 - 1)
        assert top == pieces + carried
        for heads, kv in ((32, 8), (1, 1), (64, 1), (6, 2)):
            sizes = [need(*args) for args in ((1, 1, heads, kv, dim, 385), (1, 1, heads, kv, dim, 5000), (1, 20, heads, kv, dim, 5000),
                                              (3, 20, heads, kv, dim, 5000), (3, 20, heads, kv, dim, 10 ** 6))]
            assert sizes == sorted(sizes) and sizes[-1] <= top
