"""Output rows of dsa_rotary_embed that lie on one another are refused on the
host, before anything reaches a GPU; every layout whose rows lie apart goes on to
the launch (which fails where there is no GPU)."""
import itertools

import pytest
import torch

from dsa_sparse_indexer_gb300 import _lib
from dsa_sparse_indexer_gb300 import build as B

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 4096            # a fake, 16-byte aligned "device pointer"; never dereferenced


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _lib.load()


def status(lib, T, H, D, token, head, in_place=False):
    x, out = P, P if in_place else 1 << 40
    strides = (token, head) if in_place else (H * D, D)
    return lib.dsa_rotary_embed(x, *strides, P, P, 100, 2, 0, T, H, D, 0, 0, 0, out, token, head, None, None)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T,H,D,token,head", [
    (4, 3, 64, 192, 1), (4, 3, 64, 192, 63), (4, 3, 64, 191, 64), (4, 3, 64, 1, 64), (4, 3, 64, 64, 64),
    (4, 3, 64, 128, 64), (4, 3, 64, 64, 255), (4, 3, 64, 63, 1000), (2, 1, 64, 63, 5), (1, 2, 64, 5, 63),
    (2, 2, 64, 100, 99)])
def test_rows_on_one_another_are_refused(lib, T, H, D, token, head, in_place):
    assert status(lib, T, H, D, token, head, in_place) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers")
@pytest.mark.parametrize("T,H,D,token,head", [
    (4, 3, 64, 192, 64), (4, 3, 64, 64, 256), (4, 3, 64, 1000, 64), (4, 3, 64, 70, 3000), (1, 3, 64, 0, 64),
    (1, 1, 64, 0, 0), (5, 1, 64, 64, 0), (5, 1, 64, 64, 1), (1, 2, 64, 1, 64), (2, 2, 64, 2 ** 40, 64),
    # neither dimension's rows within one step of the other's, and yet apart
    (2, 2, 8, 24, 16), (3, 2, 4, 8, 12), (2, 3, 2, 6, 4)])
def test_rows_that_lie_apart_are_not(lib, T, H, D, token, head):
    assert status(lib, T, H, D, token, head) not in (OK, INVALID, UNSUPPORTED)


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers")
def test_every_small_layout(lib):
    """Against the set of elements that each layout's rows cover."""
    for T, H, D in itertools.product((1, 2, 3, 4), (1, 2, 3), (2, 3)):
        for token, head in itertools.product(range(0, 14), range(0, 14)):
            cells = [t * token + h * head + d for t in range(T) for h in range(H) for d in range(D)]
            apart = len(set(cells)) == len(cells)
            got = status(lib, T, H, D, token, head)
            assert (got != INVALID) == apart, (T, H, D, token, head, got)
