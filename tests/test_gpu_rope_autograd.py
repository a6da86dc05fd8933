"""dsa_rotary_embed beside autograd: what it cannot record it refuses, what it
overwrites counts as overwritten, and a Function of the two directions has the
rotation's gradient."""
import numpy as np
import pytest
import torch

from oracle import rope as RO
from tests import gpu_cases as G

pytestmark = pytest.mark.gpu


def _given(T=5, H=3, D=10):
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, H, D), device="cuda", generator=gen)
    cs = RO.table(30, 8, 100.0).astype(np.float32)
    pos = np.arange(T, dtype=np.int32) * 7
    return x, pos, cs


def test_tensors_that_require_grad_are_refused():
    import dsa_sparse_indexer_gb300 as dsa
    x, pos, cs = _given()
    p, t = G.dev(pos), G.dev(cs)
    leaf = x.clone().requires_grad_()
    for given in (leaf, leaf * 2.0):
        with pytest.raises(ValueError, match="require grad"):
            dsa.rotary_embed(given, p, t)
        with pytest.raises(ValueError, match="require grad"):
            dsa.rotary_embed(given, p, t, out=given)
    with pytest.raises(ValueError, match="require grad"):
        dsa.rotary_embed(x, p, t, out=leaf)
    want = dsa.rotary_embed(x, p, t)
    with torch.no_grad():
        assert torch.equal(dsa.rotary_embed(leaf, p, t), want)
    assert torch.equal(dsa.rotary_embed(leaf.detach(), p, t), want)
    with torch.inference_mode():
        held = x.clone()
        assert torch.equal(dsa.rotary_embed(held, p, t, out=held), want)


def test_what_was_saved_for_a_backward_pass_counts_as_modified():
    import dsa_sparse_indexer_gb300 as dsa
    x, pos, cs = _given()
    w = torch.ones((), device="cuda", requires_grad=True)
    y = (x[..., :8] * w).sum()
    dsa.rotary_embed(x, G.dev(pos), G.dev(cs), out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_a_function_of_both_directions_has_the_gradient(layout):
    import dsa_sparse_indexer_gb300 as dsa
    x, pos, cs = _given()
    p, t = G.dev(pos), G.dev(cs)

    class Rotary(torch.autograd.Function):
        @staticmethod
        def forward(ctx, v):
            return dsa.rotary_embed(v, p, t, layout, first=1)

        @staticmethod
        def backward(ctx, g):
            return dsa.rotary_embed(g, p, t, layout, first=1, inverse=True)

    leaf = x.clone().requires_grad_()
    weight = torch.randn(x.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    (Rotary.apply(leaf) * weight).sum().backward()
    # the transposed rotation, value by value: 2^-23 of a pair's two values
    want = RO.rotate(weight.double().cpu().numpy(), pos, cs.astype(np.float64), layout, 1, inverse=True)
    bound = 2.0 ** -22 * float(weight.abs().max())
    assert np.abs(leaf.grad.double().cpu().numpy() - want).max() <= bound
