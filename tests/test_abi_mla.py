"""Host argument checks of the whole-context attention and the indexer's operand
entry points: every call below is refused (or has nothing to do) before anything
reaches a GPU."""
import pytest

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


def test_mla_prefill(lib):
    f = lib.dsa_mla_prefill
    #       q  qt   qh  kn  kt   kh  pe  pt  v   vt   vh  cq ck n  Tq Tk H t  sc  ca out l w  err st
    ok = (P, 384, 192, P, 512, 256, P, 64, P, 512, 256, P, P, 1, 0, 9, 2, 0, 0.1, 1, P, P, P, NULL, NULL)
    assert f(*ok) == OK                                                     # no query
    assert f(*(NULL,) * 1, *ok[1:13], 0, 4, *ok[15:]) == OK                 # no sequence
    some = list(ok)
    some[14] = 4
    check(f, some, [(0, NULL), (3, NULL), (6, NULL), (8, NULL), (11, NULL), (12, NULL), (20, NULL), (21, NULL),
                    (0, P + 8), (3, P + 2), (6, P + 8), (8, P + 8), (20, P + 8), (22, P + 4), (1, 380), (1, 0),
                    (2, 100), (2, 196), (4, 513), (5, 120), (7, 60), (9, -512), (10, 64), (13, -1), (14, -1),
                    (15, -1), (16, 0), (17, 2), (17, -1), (18, NAN), (18, INF)], INVALID)
    check(f, some, [(13, 1 << 27)], UNSUPPORTED)
    w = lib.dsa_mla_prefill_work
    assert w(4096, 4096, 1, 128) == 0                # enough items without parts
    assert w(0, 9, 1, 1) == 0 and w(9, 0, 1, 1) == 0 and w(9, 9, 0, 1) == 0 and w(9, 9, 1, 0) == 0
    need = w(16, 32768, 1, 1)
    assert need > 0 and need % (16 * 129 * 4) == 0   # parts of 16 rows: 128 values and a sum


def test_mla_decode(lib):
    f = lib.dsa_mla_decode
    #     q  kv n_slots bt reqs mb bs  qs ln mask words rows S I H scale out l w  err st
    ok = (P, P, 256, P, 2, 4, 64, P, P, P, 1, 0, 2, 1, 3, 0.1, P, P, P, NULL, NULL)
    assert f(*ok) == OK                                                     # no row
    some = list(ok)
    some[11] = 5
    none = list(some)
    none[4] = 0
    assert f(*none) == OK                                                   # no request
    check(f, some, [(0, NULL), (1, NULL), (3, NULL), (7, NULL), (8, NULL), (16, NULL), (17, NULL), (0, P + 8),
                    (1, P + 8), (16, P + 4), (18, P + 4), (2, 0), (4, -1), (5, 0), (6, 0), (10, 0), (11, -1),
                    (14, 0), (15, NAN), (15, INF)], INVALID)
    check(f, some, [(6, 48), (6, 8), (6, 65), (12, 0), (12, 65), (13, 0), (13, 1 << 30), (2, 1 << 31),
                    (14, 1 << 29)], UNSUPPORTED)
    w = lib.dsa_mla_decode_work
    assert w(64, 4, 128, 64, 64, 64) == 0            # enough items without parts
    assert w(0, 1, 1, 1, 1, 64) == 0 and w(1, 1, 1, 0, 1, 64) == 0 and w(1, 1, 1, 1, 1, 64) == 0
    need = w(1, 1, 128, 1, 512, 64)
    assert need > 0 and need % (128 * 513 * 4) == 0


def test_indexer_key_insert(lib):
    f = lib.dsa_indexer_key_insert
    #     k  kt   w  b  eps   pos cs max rot first lay slots T  S  cache n_slots err st
    ok = (P, 128, P, P, 1e-6, P, P, 64, 64, 0, 1, P, 0, 2, P, 128, NULL, NULL)
    assert f(*ok) == OK
    some = list(ok)
    some[12] = 3
    check(f, some, [(0, NULL), (2, NULL), (5, NULL), (6, NULL), (11, NULL), (14, NULL), (0, P + 8), (2, P + 4),
                    (3, P + 4), (14, P + 8), (5, P + 2), (1, 100), (1, -8), (4, -1.0), (4, NAN), (4, INF), (7, 0),
                    (8, 63), (8, 0), (8, 130), (9, 65), (9, -1), (10, 2), (12, -1), (15, 0)], INVALID)
    check(f, some, [(13, 0), (13, 65)], UNSUPPORTED)


def test_indexer_query_fp8(lib):
    f = lib.dsa_indexer_query_fp8
    #     q  qt   qh  w  fac pos cs max rot first lay T  H  q8 w8 err st
    ok = (P, 256, 128, P, 0.1, P, P, 64, 64, 0, 1, 0, 2, P, P, NULL, NULL)
    assert f(*ok) == OK
    some = list(ok)
    some[11] = 3
    check(f, some, [(0, NULL), (3, NULL), (5, NULL), (6, NULL), (13, NULL), (14, NULL), (0, P + 8), (13, P + 4),
                    (3, P + 2), (14, P + 2), (1, 100), (2, 4), (2, -8), (4, NAN), (4, INF), (7, 0), (8, 1), (9, 65),
                    (10, -1), (11, -1), (12, 0)], INVALID)
    check(f, some, [(12, 1 << 30)], UNSUPPORTED)
