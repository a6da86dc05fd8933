"""dsa_mla_prefill in fp16 where many small weights stand beside a large one.

Bounds as in test_gpu_mla_prefill, with what the type's subnormals leave of a
weight: the reference's weight is 2^7 and no larger than the largest weight, halves
of fp16's smallest step are 2^-25, so that a weight is off by 2^-11 of itself or 2^-32
of the largest, and n of them move the output by n 2^-32 max |v| at most."""
import numpy as np
import pytest
import torch

from oracle import mla_dense as MD
from tests.test_gpu_mla_prefill import inputs

pytestmark = pytest.mark.gpu


def check(q, kn, pe, v, cu_q, cu_k, scale, causal, out, lse2):
    f = lambda t: t.double().cpu().numpy()   # noqa: E731
    want, want2, size, reach = MD.prefill(f(q), f(kn), f(pe), f(v), cu_q.tolist(), cu_k.tolist(), scale, causal)
    u, d = 2.0 ** -11, 2.0 ** -16 * reach + 2.0 ** -20
    n = int((cu_k[1:] - cu_k[:-1]).max())
    tol = (u + 2 * d[..., None] + 2.0 ** -10) * size + u * np.abs(want) + n * 2.0 ** -32 * np.abs(f(v)).max()
    tol += 2.0 ** -25                            # the output's own smallest step
    assert (np.abs(f(out) - want) <= tol).all(), (np.abs(f(out) - want) / tol).max()
    seen = np.isfinite(want2)
    assert (np.abs(f(lse2) - want2)[seen] <= ((d + 2.0 ** -11) * np.log2(np.e))[seen]).all()


@pytest.mark.parametrize("depth", [12.0, 19.7, 24.0, 25.0, 27.3, 31.0])
@pytest.mark.parametrize("lq,lk,H,top", [(1, 8192, 300, -1), (1, 4000, 2, 0), (40, 3000, 200, 1500), (600, 5000, 2, -1),
                                         (700, 2100, 80, 0)])
def test_small_weights_beside_a_large_one(lq, lk, H, top, depth):
    """One key of weight 1 and value 0, the others at 2^-depth: the outputs are these."""
    import dsa_sparse_indexer_gb300 as dsa
    g = torch.Generator(device="cuda")
    g.manual_seed(lk)
    q = torch.zeros((lq, H, 192), dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    kv = torch.zeros((lk, H, 256), dtype=torch.float16, device="cuda")
    kv[..., 128:] = 0.5 + 0.5 * torch.rand((lk, H, 128), device="cuda", generator=g)
    kv[top, :, 0], kv[top, :, 128:] = depth * float(np.log(2.0)), 0.0
    pe = torch.zeros((lk, 64), dtype=torch.float16, device="cuda")
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    out, lse2 = dsa.mla_prefill(q, kv[..., :128], pe, kv[..., 128:], i(0, lq), i(0, lk), 1.0, False)
    h = sorted({0, H // 2, H - 1})               # the oracle's share
    rows = sorted({0, lq // 2, lq - 1})
    check(q[rows][:, h], kv[:, h, :128], pe, kv[:, h, 128:], i(0, len(rows)), i(0, lk), 1.0, False,
          out[rows][:, h], lse2[rows][:, h])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("gain", [0.5, 1.7, 4.0])
@pytest.mark.parametrize("lens", [[(70, 900)], [(300, 1200), (1, 500)], [(5, 7000)]])
def test_weights_of_all_sizes(lens, gain, causal):
    import dsa_sparse_indexer_gb300 as dsa
    q, kv, pe, cu_q, cu_k = inputs(lens, 2, torch.float16, seed=len(lens), gain=gain)
    args = (q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, 192.0 ** -0.5, causal)
    out, lse2 = dsa.mla_prefill(*args)
    check(*args, out, lse2)
