"""Bounds of sequences that do not ascend inside their rows: each entry is taken as
the nearest that does, so that a call gives, bit for bit, what one with those entries
gives, flags them, and leaves the rows of no sequence."""
import numpy as np
import pytest
import torch

from tests.test_gpu_mla_decode import SCALE, inputs as decode_inputs
from tests.test_gpu_mla_prefill import inputs as prefill_inputs

pytestmark = pytest.mark.gpu


def nearest(cu, T):
    return np.maximum.accumulate(np.clip(cu, 0, T))


def dev(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def descending(T, n, seed):
    """Entries mostly ascending, some below earlier ones, some outside [0, T]."""
    rng = np.random.default_rng(seed)
    cu = np.sort(rng.integers(0, T + 1, n + 1))
    for i in rng.integers(1, n + 1, max(1, n // 8)):
        cu[i] = rng.integers(-5, cu[i - 1] + 1)
    cu[n // 2] = T + 7 if seed % 2 else cu[n // 2]
    return cu


BOUNDS = [[0, 40, 20], [0, 5, 3, 9], [-3, 12, 40, 30, 60], [20, 10, 70], [0, 50, 0, 50, 0, 50], [9, 5, 3]]


@pytest.mark.parametrize("H,Tk", [(2, 90), (2, 6000), (40, 500)])
@pytest.mark.parametrize("which", range(len(BOUNDS) + 3))
def test_prefill(which, H, Tk):
    import dsa_sparse_indexer_gb300 as dsa
    T = 60
    if which < len(BOUNDS):
        cu_q = np.array(BOUNDS[which])
    else:
        cu_q = descending(T, (40, 128, 130)[which - len(BOUNDS)], seed=which)
    n = len(cu_q) - 1
    cu_k = descending(Tk, n, seed=n + which)
    q, kv, pe, _, _ = prefill_inputs([(T, Tk)], H, torch.bfloat16, seed=which)

    def call(a, b):
        out = torch.full((T, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse2, err = torch.full((T, H), 7.0, device="cuda"), dsa.new_error_flags("cuda")
        dsa.mla_prefill(q, kv[..., :128], pe, kv[..., 128:], dev(a), dev(b), SCALE, out=out, lse2=lse2, err_flags=err)
        return out, lse2, int(err)

    want = call(nearest(cu_q, T), nearest(cu_k, Tk))
    got = call(cu_q, cu_k)
    assert want[2] == 0 and got[2] == dsa.DSA_FLAG_BOUNDS
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    first, end = nearest(cu_q, T)[[0, -1]]
    assert (got[1][:first] == 7).all() and (got[1][end:] == 7).all() and not (got[1][first:end] == 7).any()


@pytest.mark.parametrize("H,length", [(2, 200), (1, 5000), (16, 300), (3, 3000), (128, 150)])
@pytest.mark.parametrize("which", range(len(BOUNDS) + 3))
def test_decode(which, H, length):
    import dsa_sparse_indexer_gb300 as dsa
    rows = 60
    if which < len(BOUNDS):
        starts = np.array(BOUNDS[which])
    else:
        starts = descending(rows, (40, 128, 130)[which - len(BOUNDS)], seed=which)
    n = len(starts) - 1
    lens = [length - 3 * i % 90 for i in range(n)]
    if length > 1000:
        lens = [length] + [60] * (n - 1)
    q, cache, table, block, _, ln, I = decode_inputs([rows] + [0] * (n - 1), lens, H, 2, 1, 64, seed=which,
                                                     cols=-(-length // 128) + 1)

    def call(a):
        out = torch.full((2, rows, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        lse2, err = torch.full((2, rows, H), 7.0, device="cuda"), dsa.new_error_flags("cuda")
        dsa.mla_decode(q, cache, table, block, dev(a), ln, I, SCALE, out=out, lse2=lse2, err_flags=err)
        return out, lse2, int(err)

    want, got = call(nearest(starts, rows)), call(starts)
    assert want[2] == 0 and got[2] == dsa.DSA_FLAG_BOUNDS
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    first, end = nearest(starts, rows)[[0, -1]]
    assert (got[1][:, :first] == 7).all() and (got[1][:, end:] == 7).all()
    assert not (got[1][:, first:end] == 7).any()
