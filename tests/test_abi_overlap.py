"""Outputs that lie on one another or on an input are refused on the host, before
anything reaches a GPU (every call below is)."""
import os
import shutil
import subprocess

import pytest

from dsa_sparse_indexer_gb300 import _lib
from dsa_sparse_indexer_gb300 import build as B

INVALID = 1
HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "dsa_sparse_indexer_gb300", "csrc")
AT = [i << 40 for i in range(1, 16)]         # fake, aligned "device pointers" far apart; never dereferenced


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _lib.load()


def check(fn, args, places, sizes, written):
    """Each written argument onto each other one: its start, and its last 16 bytes
    onto the other's start.  (Never a call that would go ahead.)"""
    for w in written:
        for other in places:
            if other == w:
                continue
            for to in (args[other], args[other] + 16 * (sizes[other] > 16), args[other] - sizes[w] + 16):
                bad = list(args)
                bad[w] = to
                assert fn(*bad) == INVALID, (w, other, hex(to))


def test_regions(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = tmp_path / "regions_check"
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", CSRC, os.path.join(HERE, "regions_check.cpp"), "-o", str(exe)],
                   check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout


def test_mla_prefill(lib):
    q, kn, pe, v, cq, ck, out, lse, work = AT[:9]
    args = [q, 384, 192, kn, 512, 256, pe, 64, v, 512, 256, cq, ck, 1, 16, 32768, 1, 0, 0.1, 1, out, lse, work, None,
            None]
    need = lib.dsa_mla_prefill_work(16, 32768, 1, 1)
    assert need > 0
    sizes = {0: 16 * 384 * 2, 3: 32768 * 512 * 2, 6: 32768 * 128, 8: 32768 * 512 * 2, 11: 8, 12: 8, 20: 16 * 256, 21: 64,
             22: need}
    check(lib.dsa_mla_prefill, args, sizes, sizes, (20, 21, 22))


def test_mla_decode(lib):
    q, kv, bt, qs, ln, mask, out, lse, work = AT[:9]
    args = [q, kv, 65536, bt, 1, 512, 64, qs, ln, mask, 1, 2, 2, 1, 16, 0.1, out, lse, work, None, None]
    need = lib.dsa_mla_decode_work(2, 2, 16, 1, 512, 64)
    assert need > 0
    sizes = {0: 2 * 16 * 1152, 1: 2 * 65536 * 1152, 3: 2 * 512 * 4, 7: 8, 8: 4, 9: 8, 16: 2 * 2 * 16 * 1024,
             17: 2 * 2 * 16 * 4, 18: need}
    check(lib.dsa_mla_decode, args, sizes, sizes, (16, 17, 18))


def test_indexer_key_insert(lib):
    k, w, b, pos, cs, slots, cache = AT[:7]
    args = [k, 136, w, b, 1e-6, pos, cs, 64, 64, 0, 1, slots, 3, 2, cache, 128, None, None]
    sizes = {0: (2 * 136 + 128) * 2, 2: 512, 3: 512, 5: 12, 6: 64 * 64 * 4, 11: 24, 14: 2 * 128 * 128}
    check(lib.dsa_indexer_key_insert, args, sizes, sizes, (14,))


def test_indexer_query_fp8(lib):
    q, w, pos, cs, q8, w8 = AT[:6]
    args = [q, 384, 136, w, 0.1, pos, cs, 64, 64, 0, 1, 4, 2, q8, w8, None, None]
    sizes = {0: (3 * 384 + 136 + 128) * 2, 3: 32, 5: 16, 6: 64 * 64 * 4, 13: 4 * 2 * 128, 14: 32}
    check(lib.dsa_indexer_query_fp8, args, sizes, sizes, (13,))
    rest = {i: n for i, n in sizes.items() if i != 3}
    check(lib.dsa_indexer_query_fp8, args, rest, sizes, (14,))
    for to in (w + 4, w - 16):                # weights themselves may be written, parts of them not
        assert lib.dsa_indexer_query_fp8(*args[:14], to, None, None) == INVALID
