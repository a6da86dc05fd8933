"""The whole-context attentions' workspaces: a call's launch splits keys as its
workspace's size says, so that the size may depend on the arguments alone, not on
which device is current, nor on whether asking it for its properties succeeds.  A
stand-in for the two calls of the CUDA runtime plays devices of other sizes."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAKE = """
static int device = 0;
void play(int d) { device = d; }
int cudaGetDevice(int* d) { *d = device; return 0; }
int cudaDeviceGetAttribute(int* value, int attribute, int d) {
  if (d == 2) return 46;                    /* unavailable */
  *value = d == 0 ? 152 : 40;
  return 0;
}
"""
ASK = """
import ctypes, sys
sys.path.insert(0, sys.argv[1])
from dsa_sparse_indexer_gb300 import _lib
lib, fake = _lib.load(), ctypes.CDLL(sys.argv[2])
seen = set()
for device in (0, 1, 2, 2, 1, 0):
    fake.play(device)
    seen.add(tuple(lib.dsa_mla_decode_work(rows, 1, 128, reqs, 512, 64) for rows, reqs in ((1, 1), (8, 2), (24, 8)))
             + tuple(lib.dsa_mla_prefill_work(tq, 32768, 1, h) for tq, h in ((16, 1), (500, 16), (700, 40))))
assert len(seen) == 1 and min(seen.pop()) > 0, seen
print("ok")
"""


def test_sizes_do_not_depend_on_the_device(tmp_path):
    from dsa_sparse_indexer_gb300 import build as B
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    B.build()
    (tmp_path / "fake.c").write_text(FAKE)
    fake = str(tmp_path / "fake.so")
    subprocess.run([cc, "-shared", "-fPIC", str(tmp_path / "fake.c"), "-o", fake], check=True)
    res = subprocess.run([sys.executable, "-c", ASK, ROOT, fake], capture_output=True, text=True,
                         env={**os.environ, "LD_PRELOAD": fake})
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout + res.stderr
