"""The rotation's angles (tests/rotary_probe.cu, on the CPU) against whole-number arithmetic: off by 1e-7 of
a radian at most, as ra.h states."""
import ctypes
import os
import random
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "sequence_blockwise_softmax_gb300", "csrc")
BITS = 400


def _pi():
    """pi * 2^BITS, off by less than 2^-300 of it: 16 atan(1/5) - 4 atan(1/239)."""
    def atan_inverse(n):
        term, total, k = (1 << BITS) // n, 0, 0
        while term:
            total += (-term if k & 1 else term) // (2 * k + 1)
            term //= n * n
            k += 1
        return total
    return 16 * atan_inverse(5) - 4 * atan_inverse(239)


PI = Fraction(_pi(), 1 << BITS)


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    out = str(tmp_path_factory.mktemp("rotary") / "rotary_probe.so")
    subprocess.run([nvcc, "-std=c++17", "-O2", "-shared", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    os.path.join(ROOT, "tests", "rotary_probe.cu"), "-o", out], check=True, capture_output=True)
    return ctypes.CDLL(out)


def worst(probe, freqs, positions):
    """The largest error in radians."""
    f, p = np.asarray(freqs, dtype=np.float32), np.asarray(positions, dtype=np.int32)
    got = np.empty(len(f), dtype=np.float32)
    ptr = lambda a: ctypes.c_void_p(a.ctypes.data)      # noqa: E731
    probe.ra_test_half_turns(ptr(f), ptr(p), ptr(got), len(f))
    turn, off = (1 << 300), 0
    half = int(turn * Fraction(1, 2))
    inverse = int(Fraction(turn) / (2 * PI))            # 1 / 2 pi, in 2^-300
    for x, n, g in zip(f, p, got):
        a, b = float(x).as_integer_ratio()
        exact = a * int(n) * inverse // b % turn
        c, d = float(g).as_integer_ratio()
        diff = (c * half // d - exact) % turn
        off = max(off, min(diff, turn - diff))
    return float(Fraction(off, turn) * 2 * PI)


@pytest.mark.parametrize("lo,hi", [(0.25, 1.0), (1e-6, 0.25), (-1.0, -1e-7), (1.0, 1e4), (-1e9, 1e9), (1e12, 3e16)])
@pytest.mark.parametrize("far", [1 << 10, 1 << 20, 1 << 29])
def test_angle(probe, lo, hi, far):
    r = random.Random(far)
    n = 20000
    assert worst(probe, [r.uniform(lo, hi) for _ in range(n)], [far - 1 - r.randrange(far // 2) for _ in range(n)]) <= 1e-7


def test_angle_of_usual_frequencies(probe):
    r = random.Random(1)
    for base in (10000.0, 500000.0, 1e6):
        freqs = [base ** (-m / 64) for m in range(64)] * 100
        assert worst(probe, freqs, [r.randrange(1 << 29) for _ in freqs]) <= 1e-7
    # one turn and its neighbours, tiny ones, none
    freqs = [1.0, 6.2831855, 3.1415927, 0.15915494, 1e-30, 1e-38, 1e-42, -1e-30, 0.0, -0.0, -6.2831855, 2.0 ** -24, 2.0 ** -72, 2.0 ** -54] * 50
    assert worst(probe, freqs, [r.randrange(1 << 29) for _ in freqs]) <= 1e-7
