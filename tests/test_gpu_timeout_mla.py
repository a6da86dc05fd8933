"""The whole-context attentions' bounded waits: in the test-only build
(build.build_stalled_copy_test) the first key blocks' barrier expects one arrival
that nothing makes.  Every copy still lands, the roles stop, nothing is written,
and the context stays usable."""
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


@pytest.mark.parametrize("T,H", [(100, 3), (700, 2), (300, 300)])
def test_prefill(stalled_lib, T, H):
    import torch

    import dsa_sparse_indexer_gb300 as dsa
    q = torch.randn((T, H, 192), device="cuda").bfloat16()
    kv = torch.randn((T, H, 256), device="cuda").bfloat16()
    pe = torch.randn((T, 64), device="cuda").bfloat16()
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out = torch.full((T, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse2 = torch.full((T, H), 7.0, device="cuda")
    err = dsa.new_error_flags("cuda")
    for _ in range(2):
        err.zero_()
        assert stalled_lib.dsa_mla_prefill(
            q.data_ptr(), q.stride(0), 192, kv.data_ptr(), kv.stride(0), 256, pe.data_ptr(), 64,
            kv[..., 128:].data_ptr(), kv.stride(0), 256, cu.data_ptr(), cu.data_ptr(), 1, T, T, H, 0, 0.07, 0,
            out.data_ptr(), lse2.data_ptr(), None, err.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()             # returns: no hang, no fault
        assert int(err.item()) == FLAG_TIMEOUT
        assert (out == 7).all() and (lse2 == 7).all()
    dsa.mla_prefill(q, kv[..., :128], pe, kv[..., 128:], cu, cu, 0.07, out=out, lse2=lse2, err_flags=err.zero_())
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and not (out == 7).all() and lse2.isfinite().all()


@pytest.mark.parametrize("rows,H,reqs", [(1, 16, 1), (1, 128, 1), (4, 128, 1), (200, 16, 200), (400, 128, 100)])
def test_decode(stalled_lib, rows, H, reqs):
    import torch

    import dsa_sparse_indexer_gb300 as dsa
    S, cols = 2, 8
    q = torch.randn((rows, H, 576), device="cuda").bfloat16()
    cache = torch.randn((S, reqs * cols * 64, 576), device="cuda").bfloat16()
    table = torch.arange(reqs * cols, device="cuda").int().view(1, reqs, cols).repeat(S, 1, 1)
    starts = torch.arange(reqs + 1, device="cuda").int() * (rows // reqs)
    lens = torch.full((reqs,), 900, dtype=torch.int32, device="cuda")
    out = torch.full((S, rows, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse2 = torch.full((S, rows, H), 7.0, device="cuda")
    err = dsa.new_error_flags("cuda")
    for _ in range(2):
        err.zero_()
        assert stalled_lib.dsa_mla_decode(
            q.data_ptr(), cache.data_ptr(), cache.shape[1], table.data_ptr(), reqs, cols, 64, starts.data_ptr(),
            lens.data_ptr(), None, 0, rows, S, 1, H, 0.07, out.data_ptr(), lse2.data_ptr(), None, err.data_ptr(),
            torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()             # returns: no hang, no fault
        assert int(err.item()) == FLAG_TIMEOUT
        assert (out == 7).all() and (lse2 == 7).all()
    dsa.mla_decode(q, cache, table, 64, starts, lens, 1, 0.07, out=out, lse2=lse2, err_flags=err.zero_())
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and not (out == 7).all() and lse2.isfinite().all()
