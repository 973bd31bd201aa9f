"""Which calls of tree attention sum a unit's key tiles in parts: all whose units can be longer than one
(tests/tree_parts_probe.cu, on the CPU)."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "sequence_blockwise_softmax_gb300", "csrc")


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    out = str(tmp_path_factory.mktemp("parts") / "tree_parts_probe.so")
    subprocess.run([nvcc, "-std=c++17", "-O2", "-shared", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"),
                    "-I", CSRC, os.path.join(ROOT, "tests", "tree_parts_probe.cu"), "-o", out], check=True, capture_output=True)
    lib = ctypes.CDLL(out)
    lib.ra_test_tree_in_parts.argtypes = [ctypes.c_longlong] * 4
    return lib


def test_no_unit_is_longer_than_a_part(probe):
    r = random.Random(1)
    part = abs(probe.ra_test_tree_in_parts(128, 1, 0, 0))
    longest, with_parts = 0, 0
    for i in range(20000):
        page = 2 ** r.randint(4, 16)
        pages = max(1, int(2 ** r.uniform(15, 22)) // page)
        n = r.choice([1, 33, 128, 500, 1024, 1024])
        max_new = r.choice([n, 1024, 10])
        window = r.choice([0, r.randint(1, 200), r.randint(100000, 140000), r.randint(part * 128 - 3000, part * 128 + 10)])
        sinks = r.choice([0, 4, r.randint(0, 300), r.randint(0, part * 128)]) if window else 0
        length = r.choice([pages * page, r.randint(0, pages * page), 10 ** 9, n, n // 2, -5])
        tiles = probe.ra_test_tree_tiles(length, n, pages, page, r.choice([1, 4, 32, 256]), max_new, window, sinks)
        if probe.ra_test_tree_in_parts(pages * page, min(max_new, n), window, sinks) < 0:
            longest = max(longest, tiles)
            assert tiles <= part, (page, pages, n, max_new, window, sinks, length)
        else:
            with_parts += 1
    assert part - 30 <= longest and with_parts > 1000


@pytest.mark.parametrize("capacity,window,sinks,parts", [
    (131072, 0, 0, False), (131072 + 16, 0, 0, True), (1 << 29, 4096, 4, False), (1 << 29, 0, 0, True),
    (1 << 29, 1 << 29, 0, True), (1 << 29, 100, 1 << 29, True), (8192, 1 << 29, 1 << 29, False),
])
def test_rule(probe, capacity, window, sinks, parts):
    assert (probe.ra_test_tree_in_parts(capacity, 60, window, sinks) > 0) == parts
