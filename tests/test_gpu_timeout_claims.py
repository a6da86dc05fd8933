"""Bounded waits that run out while items are claimed: many more items than CTAs in
the test-only build (build.build_stalled_copy_test), so that answers of the launch
control are under way when the roles stop.  The kernels return, nothing is written,
and calls of the library that follow at once on the same stream give what they gave
before."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu

FLAG_TIMEOUT = 2


@pytest.fixture(scope="module")
def stalled_lib():
    from dsa_sparse_indexer_gb300 import _lib
    from dsa_sparse_indexer_gb300 import build as B
    lib = ctypes.CDLL(B.build_stalled_copy_test())
    for name in ("dsa_mla_prefill", "dsa_mla_decode"):
        getattr(lib, name).argtypes = _lib.SIGNATURES[name][0]
    return lib


@pytest.mark.parametrize("lens,H", [([40] * 64, 16), ([600] * 12, 40)])
def test_prefill(stalled_lib, lens, H):
    import torch

    import dsa_sparse_indexer_gb300 as dsa
    T = sum(lens)
    q = torch.randn((T, H, 192), device="cuda").bfloat16()
    kv = torch.randn((T, H, 256), device="cuda").bfloat16()
    pe = torch.randn((T, 64), device="cuda").bfloat16()
    cu = torch.tensor([0] + lens, dtype=torch.int32, device="cuda").cumsum(0, dtype=torch.int32)
    args = (q, kv[..., :128], pe, kv[..., 128:], cu, cu, 0.07)
    want = dsa.mla_prefill(*args)
    for _ in range(3):
        out, lse2 = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
        err = dsa.new_error_flags("cuda")
        assert stalled_lib.dsa_mla_prefill(
            q.data_ptr(), q.stride(0), 192, kv.data_ptr(), kv.stride(0), 256, pe.data_ptr(), 64,
            kv[..., 128:].data_ptr(), kv.stride(0), 256, cu.data_ptr(), cu.data_ptr(), len(lens), T, T, H, 0, 0.07, 1,
            out.data_ptr(), lse2.data_ptr(), None, err.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        got = dsa.mla_prefill(*args)
        torch.cuda.synchronize()
        assert int(err) == FLAG_TIMEOUT and (out == 7).all() and (lse2 == 7).all()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("H,n", [(16, 1), (32, 1), (128, 1), (128, 2)])
def test_decode(stalled_lib, H, n):
    import torch

    import dsa_sparse_indexer_gb300 as dsa
    reqs, S, cols = 300, 4, 3
    rows = reqs * n
    q = torch.randn((rows, H, 576), device="cuda").bfloat16()
    cache = torch.randn((S, reqs * cols * 64, 576), device="cuda").bfloat16()
    table = torch.arange(reqs * cols, device="cuda").int().view(1, reqs, cols).repeat(S, 1, 1)
    starts = torch.arange(reqs + 1, device="cuda").int() * n
    lens = torch.full((reqs,), 700, dtype=torch.int32, device="cuda")
    args = (q, cache, table, 64, starts, lens, 1, 0.07)
    want = dsa.mla_decode(*args)
    for _ in range(3):
        out, lse2 = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
        err = dsa.new_error_flags("cuda")
        assert stalled_lib.dsa_mla_decode(
            q.data_ptr(), cache.data_ptr(), cache.shape[1], table.data_ptr(), reqs, cols, 64, starts.data_ptr(),
            lens.data_ptr(), None, 0, rows, S, 1, H, 0.07, out.data_ptr(), lse2.data_ptr(), None, err.data_ptr(),
            torch.cuda.current_stream().cuda_stream) == 0
        got = dsa.mla_decode(*args)
        torch.cuda.synchronize()
        assert int(err) == FLAG_TIMEOUT and (out == 7).all() and (lse2 == 7).all()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
