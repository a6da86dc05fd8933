"""The 8-bit attention's bounded waits: in the test-only build
(build.build_stalled_copy_test) part A of every stage expects one arrival that
nothing makes, so the scores' wait runs out.  Every copy still lands, the roles
stop, nothing is written, and the context stays usable."""
import ctypes

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

FLAG_BOUNDS, FLAG_TIMEOUT = 1, 2


@pytest.fixture(scope="module")
def stalled_lib():
    from dsa_sparse_indexer_gb300 import build as B
    from dsa_sparse_indexer_gb300 import _lib
    lib = ctypes.CDLL(B.build_stalled_copy_test())
    lib.dsa_sparse_mla_decode_fp8.argtypes = _lib.SIGNATURES["dsa_sparse_mla_decode_fp8"][0]
    return lib


@pytest.mark.parametrize("rows,H,K,split", [(1, 128, 1500, True), (1, 16, 1500, True),
                                            (3, 128, 400, True), (200, 70, 300, False),
                                            (400, 24, 300, False)])
def test_a_stalled_stage_sets_the_timeout_flag(stalled_lib, rows, H, K, split):
    import torch

    import dsa_sparse_indexer_gb300 as dsa
    from dsa_sparse_indexer_gb300 import _lib
    from tests import gpu_cases as G
    rng = np.random.default_rng(rows)
    S, n_slots = 2, 2048
    need = _lib.load().dsa_sparse_mla_decode_fp8_work(rows, S, H, K)
    assert (need > 0) == split
    q = torch.randn((rows, H, 576), device="cuda").bfloat16()
    cache = torch.randint(0, 0x78, (S, n_slots, 576), dtype=torch.uint8, device="cuda")
    scales = torch.full((S, n_slots // 64), 1 / 64, device="cuda")
    slots = G.dev(rng.integers(0, n_slots, (S, rows, K)).astype(np.int32))
    counts = G.dev(rng.integers(1, K + 1, (S, rows)).astype(np.int32))
    work = torch.zeros(max(need // 4, 4), device="cuda")
    out = torch.full((S, rows, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse2 = torch.full((S, rows, H), 7.0, device="cuda")
    err = dsa.new_error_flags("cuda")
    for _ in range(2):
        err.zero_()
        assert stalled_lib.dsa_sparse_mla_decode_fp8(
            q.data_ptr(), cache.data_ptr(), scales.data_ptr(), n_slots, 64, slots.data_ptr(),
            counts.data_ptr(), rows, S, H, K, 0.07, out.data_ptr(), lse2.data_ptr(),
            work.data_ptr() if split else None, err.data_ptr(),
            torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()             # returns: no hang, no fault
        assert int(err.item()) == FLAG_TIMEOUT
        assert (out == 7).all() and (lse2 == 7).all()
    # The context is intact: the production library attends the same slots.
    dsa.sparse_mla_decode_fp8(q, cache, scales, slots, counts, 0.07, out=out, lse2=lse2,
                              err_flags=err.zero_())
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and not (out == 7).any() and lse2.isfinite().all()
