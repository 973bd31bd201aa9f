"""The windowed attention's own tile walks, counted on the host (tests/window_probe.cu): every
pair the definition allows is met exactly once by the forward's and the dQ pass's rows and by
the dK / dV pass with its sinks' units, and no other pair is."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import window_reference as ref
from conftest import ROOT

CSRC = os.path.join(ROOT, "sequence_blockwise_softmax_gb300", "csrc")


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    out = str(tmp_path_factory.mktemp("window") / "window_probe.so")
    subprocess.run([nvcc, "-std=c++17", "-O2", "-shared", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"),
                    "-I", CSRC, os.path.join(ROOT, "tests", "window_probe.cu"), "-o", out], check=True,
                   capture_output=True)
    return ctypes.CDLL(out)


CASES = [
    # S, window, sinks, boundaries
    (1, 1, 0, None), (1, 5, 3, None), (127, 1, 0, None), (128, 128, 4, None), (129, 2, 200, None),
    (700, 100, 4, None), (700, 129, 130, None), (700, 700, 1, None), (600, 256, 0, None),
    (5000, 60, 5, None), (4097, 1000, 131, None),
    (700, 50, 4, [0, 1, 1, 300, 301, 650, 700]), (900, 33, 150, [0, 128, 256, 400, 900]),
    (5200, 77, 3, [0, 2048, 2049, 2060, 4500, 5200]), (5200, 2100, 129, [0, 10, 5200]),
    (800, 40, 6, [0, 300, 500]),                                   # tokens past the last boundary
]


@pytest.mark.parametrize("S,window,sinks,cu", CASES)
def test_every_pair_once(probe, S, window, sinks, cu):
    window, sinks = min(window, S), min(sinks, S)                   # as the entry points clip them
    ok = ref.visible(S, window, sinks, None if cu is None else cu + [S]).numpy()
    edges = None if cu is None else np.asarray(cu, dtype=np.int32)
    ptr = ctypes.c_void_p(None if cu is None else edges.ctypes.data)
    n = 0 if cu is None else len(cu) - 1
    for rows in (256, 128):
        cnt = np.zeros((S, S), dtype=np.int32)
        probe.ra_test_window_rows(S, window, sinks, ptr, n, rows, ctypes.c_void_p(cnt.ctypes.data))
        assert np.array_equal(cnt, ok.astype(np.int32)), rows
    for slot_bytes in (0, 4 << 20):         # the second makes the sinks' chunks longer
        cnt = np.zeros((S, S), dtype=np.int32)
        assert probe.ra_test_window_cols(S, window, sinks, ptr, n, slot_bytes, ctypes.c_void_p(cnt.ctypes.data)) == 0
        assert np.array_equal(cnt, ok.astype(np.int32))


@pytest.mark.parametrize("units,blocks", [(1, 2), (75, 150), (76, 152), (77, 77), (152, 152), (153, 153), (4096, 4096)])
def test_units_and_halves(probe, units, blocks):
    cnt = np.zeros(units * 256, dtype=np.int32)
    assert probe.ra_test_window_units(units, 152, ctypes.c_void_p(cnt.ctypes.data)) == blocks
    assert (cnt == 1).all()


def test_reference_gradients_are_differences():
    """The formula the kernels are held to, against central differences of the 64-bit forward."""
    g = torch.Generator().manual_seed(3)
    L, H, Hkv, d, scale = 13, 4, 2, 8, 0.31
    q, k, v, do = (torch.randn((1, L, h, d), generator=g, dtype=torch.float64) for h in (H, Hkv, Hkv, H))
    ok = ref.visible(L, 4, 2, [0, 5, 13])

    def loss(a, b, c):
        return (ref.forward(a, ref.expand_kv(b, H), ref.expand_kv(c, H), ok, scale)[0] * do).sum()

    o, lse, _ = ref.forward(q, ref.expand_kv(k, H), ref.expand_kv(v, H), ok, scale)
    grads, _ = ref.backward(q, ref.expand_kv(k, H), ref.expand_kv(v, H), o, do, lse, ok, scale, Hkv)
    h = 1e-5
    for i in range(3):
        for _ in range(6):
            step = torch.randn((q, k, v)[i].shape, generator=g, dtype=torch.float64)
            up, down = [q, k, v], [q, k, v]
            up[i], down[i] = up[i] + h * step, down[i] - h * step
            diff = (loss(*up) - loss(*down)) / (2 * h)
            assert abs(diff - (grads[i] * step).sum()) < 1e-7 * max(1.0, abs(diff))


FAKE = 0x10000


def _fwd(lib, **kw):
    a = dict(q=FAKE, cu=None, n=0, B=1, L=1024, H=4, Hkv=2, d=128, W=100, sinks=4, scale=0.0, flags=0, ws=FAKE, wsb=256)
    a.update(kw)
    return lib.ra_window_attn_fwd(a["q"], FAKE, FAKE, FAKE, FAKE, a["cu"], a["n"], a["B"], a["L"], a["H"], a["Hkv"],
                                  a["d"], a["W"], a["sinks"], a["scale"], a["flags"], a["ws"], a["wsb"], None)


BAD = [
    (dict(W=0), 1), (dict(W=-1), 1), (dict(sinks=-1), 1), (dict(Hkv=3), 2), (dict(Hkv=0), 2), (dict(d=96), 3),
    (dict(flags=1), 1), (dict(flags=4), 1), (dict(scale=float("inf")), 1), (dict(q=0), 1), (dict(q=FAKE + 8), 4),
    (dict(wsb=128), 1), (dict(ws=0), 1), (dict(n=2), 1), (dict(cu=FAKE, n=0), 2), (dict(cu=FAKE, n=2, B=2), 2),
    (dict(cu=FAKE + 2, n=2), 4), (dict(L=1 << 30), 3), (dict(B=-1), 2),
    (dict(B=1 << 20, H=1 << 20, Hkv=1), 3),
]


@pytest.mark.parametrize("kw,status", BAD)
def test_forward_refuses(ralib, kw, status):
    assert _fwd(ralib.lib(), **kw) == status
    assert ralib.lib().ra_last_error().decode()


@pytest.mark.parametrize("kw,status", BAD + [(dict(flags=16), 1)])
def test_backward_refuses(ralib, kw, status):
    a = dict(q=FAKE, cu=None, n=0, B=1, L=1024, H=4, Hkv=2, d=128, W=100, sinks=4, scale=0.0, flags=0, ws=FAKE,
             wsb=1 << 40)
    a.update(kw)
    st = ralib.lib().ra_window_attn_bwd(a["q"], *[FAKE] * 8, a["cu"], a["n"], a["B"], a["L"], a["H"], a["Hkv"],
                                        a["d"], a["W"], a["sinks"], a["scale"], a["flags"], a["ws"], a["wsb"], None)
    assert st == status


def test_empty_calls_launch_nothing(ralib):
    assert _fwd(ralib.lib(), L=0, q=0, ws=0) == 0
    assert _fwd(ralib.lib(), B=0, q=0, ws=0) == 0


def test_backward_workspace(ralib):
    f = ralib.ra_window_attn_bwd_workspace_bytes
    r = lambda n: (n + 255) // 256 * 256
    assert f(1, 1000, 4, 2, 64, 100) == 256 + r(16000)
    assert f(1, 1000, 4, 2, 64, 1000, 8) == 256 + r(16000)          # no query past a window of L
    # chunks of 512 queries, one more for each sequence, and each sequence's own part
    assert f(1, 5000, 4, 2, 64, 100, 8) == 256 + r(80000) + 2 * 2 * (10 + 1) * 8 * 64 * 4
    assert f(1, 5000, 4, 2, 64, 100, 8, n_seqs=5) == 256 + r(80000) + 2 * 2 * (15 + 6) * 8 * 64 * 4
    assert f(1, 5000, 4, 2, 64, 1000, 8) == 256 + r(80000) + 2 * 2 * (5 + 1) * 8 * 64 * 4
    # many sinks and heads: longer chunks keep the partial gradients near 32 MiB
    assert f(2, 32768, 8, 8, 128, 1, 129) - 256 - 4 * 2 * 32768 * 8 <= 33 << 20
    assert f(1, 1 << 29, 1 << 9, 1 << 9, 128, 1, 1 << 29) == 0      # would leave 64 bits
    assert f(1, 128, 1 << 20, 1 << 20, 128, 1, 128, n_seqs=(1 << 31) - 1) == 0
    assert f(1, 5000, 4, 2, 96, 100, 8) == 0 and f(1, 5000, 4, 2, 64, 0, 8) == 0


def test_binding_refuses_host_tensors(ralib):
    x = torch.zeros((1, 8, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ralib.ra_window_attn_fwd(x, x, x, x, torch.zeros(1, 2, 8), 1, 8, 2, 2, 64, 4,
                                 workspace=torch.zeros(256, dtype=torch.uint8))
