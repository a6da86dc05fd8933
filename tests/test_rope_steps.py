"""Host-only check of the rotation tables' angles per position
(csrc/rope_steps.h): 2^64 w_i / (2 pi) rounded once, against the definition in
80-digit decimal arithmetic.

Tolerance: half a unit for the rounding, and the arithmetic's 2^-80 of a value
that is at most 2^61.4, so below 2^-18 of a unit (as much as a relative error of
2^-80 at the largest step); 2^-10 leaves room for the few operations of each."""
import os
import random
import shutil
import subprocess
from decimal import Decimal, getcontext

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "dsa_sparse_indexer_gb300", "csrc")
TWO_PI = Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257241799725606965068")
NONE, LINEAR, NTK, YARN = range(4)


def _exact(rot, base, kind, factor, orig, fast, slow):
    import math
    getcontext().prec = 80
    b, f, d = Decimal(base), Decimal(factor), Decimal(rot)
    ln = b.ln()
    if kind == NTK and rot > 2:
        ln += f.ln() * d / (d - 2)
    if kind == YARN:
        index = lambda turns: rot * math.log(orig / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        low = max(math.floor(index(fast)), 0)
        span = max(min(math.ceil(index(slow)), rot - 1) - low, 0.001)
    out = []
    for i in range(rot // 2):
        w = (-2 * Decimal(i) / d * ln).exp()
        if kind == LINEAR:
            w /= f
        if kind == YARN:
            r = min(max(Decimal(i - low) / Decimal(span), Decimal(0)), Decimal(1))
            w = w * (1 - r) + w / f * r
        out.append(w / TWO_PI * 2 ** 64)
    return out


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = tmp_path_factory.mktemp("steps") / "rope_steps_check"
    subprocess.run([cxx, "-O3", "-std=c++17", "-I", CSRC, os.path.join(HERE, "rope_steps_check.cpp"),
                    "-o", str(exe)], check=True)
    return str(exe)


def _cases():
    rng = random.Random(1)
    cases = [(2, 1e4, k, 3.0, 4096, 32.0, 1.0) for k in range(4)]
    cases += [(256, 1e4, NONE, 1.0, 4096, 32.0, 1.0), (4, 1.0000001, NONE, 1.0, 1, 32.0, 1.0),
              (64, 1e4, YARN, 32.0, 4096, 32.0, 1.0), (64, 1e4, YARN, 1.0, 4096, 32.0, 1.0),
              (8, 1e4, YARN, 4.0, 1, 2.0, 1.0), (8, 1e4, YARN, 4.0, 2 ** 31 - 1, 1.5, 1.5),
              (4, 1e4, NTK, 1e6, 1, 1.0, 1.0), (256, 1e200, NTK, 1e100, 1, 1.0, 1.0)]
    for _ in range(60):
        kind = rng.randrange(4)
        cases.append((2 * rng.randint(1, 128), rng.choice([1e4, 5e5, 1e6, 10 ** rng.uniform(0.01, 9)]), kind,
                      rng.choice([1.0, 8.0, rng.uniform(1, 40)]), rng.choice([512, 4096, 8192, 131072]),
                      32.0, rng.choice([1.0, 0.5])))
    return cases


def test_steps_are_the_exact_ones_rounded(program):
    cases = _cases()
    text = "".join(f"{r} {float(b).hex()} {k} {float(f).hex()} {o} {float(x).hex()} {float(y).hex()}\n"
                   for r, b, k, f, o, x, y in cases)
    out = subprocess.run([program], input=text, capture_output=True, text=True, check=True).stdout
    lines = out.splitlines()
    assert len(lines) == len(cases)
    for case, line in zip(cases, lines):
        got = [int(v) for v in line.split()]
        for i, (g, want) in enumerate(zip(got, _exact(*case), strict=True)):
            assert abs(Decimal(g) - want) <= Decimal(0.5) + Decimal(2) ** -10, (case, i, g, want)
