"""GPU parity of dsa_sparse_mla_decode_fp8 on both sides of the numbers of
(row, head group) pairs that are split over eight, four and two CTAs, against the
fp64 softmax, with the bounds of tests/test_gpu_fp8_mixed_scales.py."""
import numpy as np
import pytest

from tests.test_gpu_fp8_mixed_scales import _codes, _compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,H", [(7, 128), (8, 128), (9, 128), (15, 64), (16, 48), (18, 128), (19, 128),
                                    (36, 64), (37, 20), (38, 128), (39, 128), (76, 64), (77, 64)])
@pytest.mark.parametrize("K", [2048, 1100])
def test_every_number_of_parts(rows, H, K):
    rng = np.random.default_rng(rows)
    n, block = 4096, 64
    scales = np.exp2(rng.integers(-8, -4, n // block)).astype(np.float64)
    q = rng.standard_normal(576) * 2.0
    _compare(rows, H, q, _codes(rng, n), scales, block, rng.permutation(n)[:K])


def test_captured_and_replayed():
    """A split call in a graph, replayed with other inputs: the bits of a call."""
    import torch

    import dsa_sparse_indexer_gb300 as dsa
    gen = torch.Generator(device="cuda").manual_seed(3)
    rows, H, K, n = 9, 128, 2048, 8192
    cache = torch.randint(0, 0x78, (1, n, 576), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.full((1, n // 64), 2.0 ** -9, device="cuda")
    make = lambda: (torch.randn((rows, H, 576), device="cuda", generator=gen).bfloat16(),      # noqa: E731
                    torch.randint(0, n, (1, rows, K), dtype=torch.int32, device="cuda", generator=gen),
                    torch.randint(0, K + 1, (1, rows), dtype=torch.int32, device="cuda", generator=gen))
    calls = [make(), make()]
    alone = [dsa.sparse_mla_decode_fp8(q, cache, scales, sl, ct, 0.07) for q, sl, ct in calls]
    held = [t.clone() for t in calls[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse2 = dsa.sparse_mla_decode_fp8(held[0], cache, scales, held[1], held[2], 0.07)
    for k in (1, 0):
        for t, new in zip(held, calls[k]):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, alone[k][0]) and torch.equal(lse2, alone[k][1])
