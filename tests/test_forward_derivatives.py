"""Calls that autograd does not see refuse tensors that carry a tangent (forward-mode
derivatives), whether gradients are recorded or not, as they refuse those that require
grad."""
import pytest
import torch
from torch.autograd import forward_ad


def test_tangents_are_found():
    from dsa_sparse_indexer_gb300 import ops
    x, y = torch.zeros(3), torch.zeros(3, dtype=torch.int32)
    ops._no_grad(x, None, y)
    with forward_ad.dual_level():
        ops._no_grad(x, None, y)                 # none carries one
        dual = forward_ad.make_dual(x, torch.ones(3))
        for enabled in (False, True):
            with torch.set_grad_enabled(enabled), pytest.raises(ValueError):
                ops._no_grad(y, dual)
    ops._no_grad(x, y)
    with pytest.raises(ValueError):
        ops._no_grad(x, torch.zeros(3, requires_grad=True))


@pytest.mark.gpu
def test_calls_refuse_tangents():
    import dsa_sparse_indexer_gb300 as dsa
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    cs, w = dsa.rope_table(8, 64), torch.ones(128, device="cuda")
    with torch.no_grad(), forward_ad.dual_level():
        dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))   # noqa: E731
        for call in (lambda f: dsa.mla_prefill(f(bf(2, 1, 192)), bf(2, 1, 128), bf(2, 64), bf(2, 1, 128), i(0, 2), i(0, 2), 1.0),
                     lambda f: dsa.mla_prefill(bf(2, 1, 192), bf(2, 1, 128), bf(2, 64), f(bf(2, 1, 128)), i(0, 2), i(0, 2), 1.0),
                     lambda f: dsa.mla_decode(f(bf(1, 1, 576)), bf(1, 64, 576), i(0).view(1, 1, 1), 64, i(0, 1), i(1), 1, 1.0),
                     lambda f: dsa.indexer_key_insert(bf(1, 128), f(w), None, 1e-6, i(0), cs, i(0).view(1, 1),
                                                      torch.zeros((1, 64, 128), dtype=torch.uint8, device="cuda")),
                     lambda f: dsa.indexer_query_fp8(f(bf(1, 1, 128)), torch.ones((1, 1), device="cuda"), i(0), cs),
                     lambda f: dsa.rotary_embed(f(bf(1, 64)), i(0), cs)):
            call(lambda t: t)
            with pytest.raises(ValueError, match="tangent"):
                call(dual)
