"""The paged attention's arithmetic at the largest sizes a call may have, on the host
(tests/paged_sizes_probe.cu)."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "sequence_blockwise_softmax_gb300", "csrc")


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    out = str(tmp_path_factory.mktemp("sizes") / "paged_sizes_probe.so")
    subprocess.run([nvcc, "-std=c++17", "-O2", "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-fsanitize=signed-integer-overflow",
                    "-Xcompiler", "-fsanitize-undefined-trap-on-error", "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(ROOT, "tests", "paged_sizes_probe.cu"), "-o", out], check=True,
                   capture_output=True)
    lib = ctypes.CDLL(out)
    lib.path = out
    return lib


@pytest.mark.parametrize("n,chunks", [
    (0, [1]), (1, [0]), (1, [1]), (1, [1 << 25]), (1000, [0, 3, 1, 0, 70]),
    ((1 << 23) - 1, [1]), (1 << 23, [1]), (1 << 23, [1 << 16]), (1 << 24, [1]), (1 << 24, [1 << 15]), (1 << 24, [0, 1 << 16]),
    (1 << 14, [1 << 25]),                       # 2^14 sequences of 2^29 keys: 2^43 in all
])
def test_every_sequence_and_chunk_counts(probe, n, chunks):
    out = (ctypes.c_int64 * 2)()
    probe.ra_test_paged_tally(ctypes.c_int64(n), (ctypes.c_int * len(chunks))(*chunks), len(chunks), out)
    whole, rest = divmod(n, len(chunks))
    some = lambda f: whole * sum(map(f, chunks)) + sum(map(f, chunks[:rest]))
    assert list(out) == [some(lambda c: c > 0), some(lambda c: c)]


@pytest.mark.parametrize("pairs,keys,n,ctas", [
    (1 << 40, 1 << 29, 1 << 24, 304),           # 2^24 sequences of 2^16 heads over 2^29 keys: 2^65 chunks
    (1 << 36, 1 << 29, 1 << 24, 304), (152, 1 << 29, 1, 304), (1, 1 << 29, 1, 304), (1, 0, 1, 2), (153, 20000, 153, 304),
    (300, 20000, 300, 304), (400, 500, 400, 400), (3, 10000, 3, 304), (1, 10000, 1, 157),
])
def test_grid_of_any_size(probe, pairs, keys, n, ctas):
    """In a process of its own: a sum that leaves 64 bits ends it."""
    code = "import ctypes, sys; i = ctypes.c_int64; p = ctypes.CDLL(%r); print(p.ra_test_paged_ctas(i(%d), i(%d), i(%d)))"
    r = subprocess.run([sys.executable, "-c", code % (probe.path, pairs, keys, n)], capture_output=True, text=True)
    assert r.returncode == 0, r.returncode
    assert int(r.stdout) == ctas
