"""Host argument checks of the rotation and 8-bit cache entry points: every
call below is refused (or has nothing to do) before anything reaches a GPU."""
import pytest
import torch

from dsa_sparse_indexer_gb300 import _lib
from dsa_sparse_indexer_gb300 import build as B

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 4096            # a fake, 16-byte aligned "device pointer"; never dereferenced
NULL = None
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _lib.load()


def check(fn, ok, bad, status):
    for i, value in bad:
        args = list(ok)
        args[i] = value
        assert fn(*args) == status, (i, value)


def test_rope_table(lib):
    f = lib.dsa_rope_table
    #     max_pos rot base scaling factor orig fast slow amp table stream
    ok = (0, 64, 1e4, 3, 4.0, 4096, 32.0, 1.0, 1.0, NULL, NULL)
    assert f(*ok) == OK
    check(f, (8, *ok[1:9], P, NULL),
          [(0, -1), (1, 63), (1, 0), (2, 1.0), (2, INF), (2, NAN), (3, -1), (3, 4), (4, 0.5),
           (4, NAN), (4, INF), (5, 0), (6, 0.5), (7, 0.0), (7, NAN), (6, INF), (8, NAN),
           (9, NULL), (9, P + 2)], INVALID)
    check(f, (8, *ok[1:9], P, NULL), [(1, 258)], UNSUPPORTED)
    # a scaling other than YaRN does not read its arguments
    assert f(0, 64, 1e4, 0, 1.0, 0, 0.0, 0.0, 1.0, NULL, NULL) == OK


def test_rotary_embed(lib):
    f = lib.dsa_rotary_embed
    #     x  xt   xh   pos tab max rot first T H D  type layout inv out ot  oh  err stream
    ok = (P, 192, 64, P, P, 100, 32, 16, 0, 3, 64, 0, 0, 0, 2 * P, 192, 64, NULL, NULL)
    assert f(*ok) == OK                                                     # no token
    assert f(NULL, 0, 0, NULL, NULL, 100, 32, 16, 5, 0, 64, 0, 0, 0, NULL, 0, 0, NULL, NULL) == OK
    some = list(ok)
    some[8] = 4
    check(f, some, [(0, NULL), (3, NULL), (4, NULL), (14, NULL), (0, P + 1), (14, P + 1),
                    (4, P + 2), (1, -1), (2, -1), (15, -1), (16, -1), (5, 0), (6, 31), (6, 0),
                    (7, -1), (7, 33), (8, -1), (9, -1), (10, 0), (11, 3), (11, -1), (12, 2),
                    (15, 0), (16, 0)], INVALID)
    aliased = list(some)
    aliased[14], aliased[15] = P, 200                # in place with other strides
    assert f(*aliased) == INVALID
    fp32 = list(some)
    fp32[11], fp32[0] = 2, P + 2
    assert f(*fp32) == INVALID
    check(f, some, [(10, 1025)], UNSUPPORTED)
    huge = list(some)
    huge[8], huge[9] = 1 << 16, 1 << 15
    assert f(*huge) == UNSUPPORTED


def test_kv_cache_insert_fp8(lib):
    f = lib.dsa_kv_cache_insert_fp8
    #     kv kpe slots T cache scales n_slots block work err stream
    ok = (NULL, NULL, NULL, 0, NULL, NULL, 128, 64, NULL, NULL, NULL)
    assert f(*ok) == OK
    some = (P, P, P, 4, P, P, 128, 64, NULL, NULL, NULL)
    check(f, some, [(0, NULL), (1, NULL), (2, NULL), (4, NULL), (5, NULL), (0, P + 8), (1, P + 4),
                    (4, P + 8), (3, -1), (6, 0), (6, 100), (7, 0)], INVALID)
    check(f, some, [(6, 2 ** 31)], UNSUPPORTED)
    assert f(P, P, P, 4, P, P, 2050, 1025, NULL, NULL, NULL) == UNSUPPORTED
    assert f(P, P, P, 513, P, P, 128, 64, NULL, NULL, NULL) == INVALID      # needs work


def test_sparse_mla_decode_fp8(lib):
    f = lib.dsa_sparse_mla_decode_fp8
    #     q  cache scales n_slots block slots counts rows S H K scale out lse work err stream
    ok = (NULL, NULL, NULL, 128, 64, NULL, NULL, 0, 2, 16, 512, 0.1, NULL, NULL, NULL, NULL, NULL)
    assert f(*ok) == OK
    some = (P, P, P, 128, 64, P, P, 3, 2, 16, 512, 0.1, P, P, NULL, NULL, NULL)
    check(f, some, [(0, NULL), (1, NULL), (2, NULL), (5, NULL), (6, NULL), (12, NULL), (13, NULL),
                    (0, P + 8), (1, P + 8), (12, P + 8), (14, P + 4), (3, 0), (3, 100), (4, 0),
                    (7, -1),
                    (9, 0), (10, 0), (11, INF), (11, NAN)], INVALID)
    check(f, some, [(8, 0), (8, 65), (3, 2 ** 32), (7, 2 ** 30), (10, 2 ** 30 + 1)], UNSUPPORTED)


def test_sparse_mla_decode_fp8_work(lib):
    f = lib.dsa_sparse_mla_decode_fp8_work
    assert f(64, 4, 128, 2048) == 0                 # more pairs than SMs
    one = f(1, 1, 128, 2048)
    assert one == 2 * 8 * (64 * 512 + 256) * 4      # two head groups, eight parts
    assert f(1, 1, 16, 2048) == one // 2
    assert f(1, 1, 128, 300) == 0                   # three tiles: not worth a merge
    for bad in ((0, 1, 128, 2048), (1, 0, 128, 2048), (1, 65, 128, 2048), (1, 1, 0, 2048),
                (1, 1, 128, 0)):
        assert f(*bad) == 0
    assert f(2 ** 31 - 1, 64, 2 ** 31 - 1, 2 ** 31 - 1) == 0


def test_binding_refusals():
    import dsa_sparse_indexer_gb300 as dsa
    x = torch.zeros(4, 2, 64)
    pos, tab = torch.zeros(4, dtype=torch.int32), torch.zeros(8, 64)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.rotary_embed(x, pos, tab)
    with pytest.raises(ValueError, match="layout"):
        dsa.rotary_embed(x, pos, tab, layout="neox")
    with pytest.raises(TypeError, match="bf16, fp16 or fp32"):
        dsa.rotary_embed(x.double(), pos, tab)
    with pytest.raises(TypeError, match="Tensor"):
        dsa.rotary_embed(None, pos, tab)
    with pytest.raises(ValueError, match="scaling"):
        dsa.rope_table(8, 64, scaling="other")
    with pytest.raises(ValueError, match="CUDA"):
        dsa.rope_table(8, 64, out=tab)
    with pytest.raises(ValueError, match="negative"):
        dsa.rope_table(-8, 64)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.kv_cache_insert_fp8(torch.zeros(4, 512).bfloat16(), torch.zeros(4, 64).bfloat16(),
                                pos, torch.zeros(64, 576, dtype=torch.uint8), torch.zeros(1))
    with pytest.raises(ValueError, match="CUDA"):
        dsa.sparse_mla_decode_fp8(torch.zeros(1, 2, 576).bfloat16(),
                                  torch.zeros(1, 64, 576, dtype=torch.uint8), torch.zeros(1, 1),
                                  torch.zeros(1, 1, 8, dtype=torch.int32),
                                  torch.zeros(1, 1, dtype=torch.int32), 0.1)
