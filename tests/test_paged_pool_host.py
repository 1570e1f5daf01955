"""Pools that a plan cannot write while it reads them are refused before anything is launched (no GPU needed)."""
import ctypes as C

import pytest
import torch

# the addresses are made up: a library that did not refuse them must find no device to follow them on
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: run without a GPU")


@pytest.fixture(scope="module")
def lib():
    from dense_decoder_block_gb300 import _native, build
    return _native.load(build.build())


@pytest.mark.parametrize("words", [-1, 1])
def test_overlapping_pools_are_refused(lib, words):
    P, at = C.c_void_p(1 << 20), C.c_void_p((1 << 20) + 4 * words)
    assert lib.llama_paged_plan(P, P, 2, 3, 16, 8, P, P, at, P, 4, P, None, None) == -1
    assert lib.llama_paged_release(P, P, 2, 16, 8, P, P, at, P, 4, None, None) == -1
