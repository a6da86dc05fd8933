"""Tokens that dsa_rotary_embed carries: a position outside the table leaves its
token bit for bit as it is, whatever the values."""
import numpy as np
import pytest
import torch

from oracle import rope as RO
from tests import gpu_cases as G

pytestmark = pytest.mark.gpu

BITS = {torch.bfloat16: torch.int16, torch.float16: torch.int16, torch.float32: torch.int32}


@pytest.mark.parametrize("dtype", list(BITS))
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T,H,D,rot,first", [(4, 2, 64, 64, 0), (4, 3, 37, 22, 5), (4, 2, 34, 20, 2),
                                             (3000, 9, 64, 64, 0), (3000, 8, 66, 62, 2)])
@pytest.mark.parametrize("inverse", [False, True])
def test_infinities_nan_and_zeros_are_carried(dtype, layout, T, H, D, rot, first, inverse):
    import dsa_sparse_indexer_gb300 as dsa
    gen = torch.Generator(device="cuda").manual_seed(D)
    x = torch.randn((T, H, D), device="cuda", generator=gen).to(dtype)
    special = torch.tensor([float("inf"), -float("inf"), float("nan"), -0.0, 0.0, 1.0, 3e-38, 65504.0],
                           device="cuda").to(dtype)
    pick = torch.randint(0, 8, x.shape, device="cuda", generator=gen)
    x = torch.where(torch.rand(x.shape, device="cuda", generator=gen) < 0.5, special[pick], x)
    out_of = np.arange(T) % 4 != 1
    pos = np.where(out_of, np.array([10, 3, -1, 2 ** 31 - 1])[np.arange(T) % 4], 3).astype(np.int32)
    cs = G.dev(RO.table(10, rot, 10000.0).astype(np.float32))
    err = dsa.new_error_flags("cuda")
    got = dsa.rotary_embed(x, G.dev(pos), cs, layout, first, inverse, err_flags=err)
    assert int(err.item()) == dsa.DSA_FLAG_BOUNDS
    carried = G.dev(out_of)
    assert torch.equal(got[carried].view(BITS[dtype]), x[carried].view(BITS[dtype]))
    # the tokens between them turn as they do alone
    alone = dsa.rotary_embed(x[~carried], G.dev(pos[~out_of]), cs, layout, first, inverse)
    assert torch.equal(got[~carried].view(BITS[dtype]), alone.view(BITS[dtype]))
