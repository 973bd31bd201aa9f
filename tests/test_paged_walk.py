"""The paged attention's own units, splits and walks, counted on the host (tests/paged_probe.cu),
and what its entry points refuse."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from conftest import ROOT

CSRC = os.path.join(ROOT, "sequence_blockwise_softmax_gb300", "csrc")


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    out = str(tmp_path_factory.mktemp("paged") / "paged_probe.so")
    subprocess.run([nvcc, "-std=c++17", "-O2", "-shared", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"),
                    "-I", CSRC, os.path.join(ROOT, "tests", "paged_probe.cu"), "-o", out], check=True,
                   capture_output=True)
    return ctypes.CDLL(out)


CASES = [
    # new tokens, lengths, page, max_pages, group, unit_tokens, window, sinks, splits
    ([1], [1], 16, 1, 4, 64, 0, 0, 1),
    ([1, 1, 1], [5, 300, 4000], 16, 256, 8, 32, 0, 0, 19),
    ([0, 3, 0, 200, 1], [7, 3, 0, 3000, 513], 32, 100, 5, 50, 0, 0, 4),
    ([257], [2000], 256, 8, 1, 256, 100, 4, 3),
    ([64, 65, 63], [64, 1900, 2048], 128, 16, 2, 64, 1700, 130, 2),
    ([10, 1], [3000, 3000], 64, 50, 128, 2, 33, 1, 8),
    ([5, 4], [3, 4], 16, 4, 1, 256, 0, 0, 1),                    # more new tokens than length: negative positions
    ([4], [100], 16, 4, 1, 256, 0, 0, 1),                        # longer than its table row
]


@pytest.mark.parametrize("new,lens,page,max_pages,group,unit,window,sinks,splits", CASES)
@pytest.mark.parametrize("tail,share", [(0, 0), (5, 0), (0, 1), (0, 0.4)])
def test_every_pair_once(probe, new, lens, page, max_pages, group, unit, window, sinks, splits, tail, share):
    n, T = len(new), sum(new) + tail
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    sl = np.asarray(lens, dtype=np.int32)
    cap = max_pages * page
    cnt = np.zeros((T, cap), dtype=np.int32)
    loaded = np.zeros((n, max_pages), dtype=np.int32)
    seen = ctypes.c_int(0)
    p = lambda a: ctypes.c_void_p(a.ctypes.data)
    assert probe.ra_test_paged(p(sl), p(cu), n, T, max_pages, page, group, 1, unit, max(new), window, sinks, splits,
                               int(share * 1024 / splits), p(cnt), p(loaded), ctypes.byref(seen)) == 0
    want = np.zeros_like(cnt)
    key = np.arange(cap)
    for s in range(n):
        length = min(lens[s], cap)
        for i in range(new[s]):
            pos = length - new[s] + i
            ok = key <= pos
            if window:
                ok &= (key > pos - window) | (key < sinks)
            want[cu[s] + i] = ok
        held = -(-length // page)
        assert not loaded[s, held:].any()
        if new[s] and window and length > 4 * (window + unit + sinks + page + 256):
            assert loaded[s].sum() < held
    assert np.array_equal(cnt, want)
    cnt[:] = 0
    assert probe.ra_test_paged_chunks(p(sl), p(cu), n, T, max_pages, page, max(new), window, sinks, p(cnt)) == 0
    assert np.array_equal(cnt, want)
    if splits > 1 and max(min(x, cap, window or cap) for x in lens) >= 1536:
        assert seen.value > 1


def test_bad_boundaries_stay_inside(probe):
    """cu_q of any content: no row outside [0, T) and no page outside the table row."""
    rng = np.random.RandomState(1)
    for _ in range(200):
        n, T, page, max_pages = rng.randint(1, 9), rng.randint(1, 400), 16, rng.randint(1, 40)
        cu = rng.randint(-50, 500, n + 1).astype(np.int32)
        sl = rng.randint(-50, 1000, n).astype(np.int32)
        cnt = np.zeros((T, max_pages * page), dtype=np.int32)
        loaded = np.zeros((n, max_pages), dtype=np.int32)
        seen = ctypes.c_int(0)
        p = lambda a: ctypes.c_void_p(a.ctypes.data)
        assert probe.ra_test_paged(p(sl), p(cu), n, T, max_pages, page, 4, 1, 64, int(rng.randint(1, 300)),
                                   int(rng.randint(0, 200)), int(rng.randint(0, 200)), 4, int(rng.randint(0, 257)),
                                   p(cnt), p(loaded),
                                   ctypes.byref(seen)) == 0
        assert probe.ra_test_paged_chunks(p(sl), p(cu), n, T, max_pages, page, int(rng.randint(1, 300)), 50, 20, p(cnt)) == 0


FAKE = 0x10000


def _fwd(lib, **kw):
    a = dict(q=FAKE, k=FAKE, table=FAKE, o=FAKE, lse=FAKE, T=64, n=4, H=8, Hkv=2, d=128, n_pages=100, page=16,
             pstride=16 * 2 * 128, max_pages=20, qs=1024, new=16, len=300, W=0, sinks=0, scale=0.0, flags=0, ws=FAKE,
             wsb=1 << 40)
    a.update(kw)
    return lib.ra_paged_attn_fwd(a["q"], a["k"], FAKE, a["table"], FAKE, FAKE, a["o"], a["lse"], a["T"], a["n"], a["H"],
                                 a["Hkv"], a["d"], a["n_pages"], a["page"], a["pstride"], a["max_pages"], a["qs"],
                                 a["new"], a["len"], a["W"], a["sinks"], a["scale"], a["flags"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=80), 3), (dict(Hkv=3), 2), (dict(Hkv=0), 2), (dict(H=129, Hkv=1, qs=129 * 128, pstride=1 << 20), 3),
    (dict(page=24), 3), (dict(page=8), 3), (dict(page=0), 3), (dict(pstride=16 * 2 * 128 - 8), 2),
    (dict(pstride=16 * 2 * 128 + 4), 4), (dict(qs=1016), 2), (dict(qs=1028), 4), (dict(T=-1), 2), (dict(n=-1), 2),
    (dict(max_pages=1 << 27), 3), (dict(W=-1), 1), (dict(sinks=-1), 1), (dict(scale=float("nan")), 1), (dict(flags=4), 1),
    (dict(q=0), 1), (dict(k=FAKE + 8), 4), (dict(table=0), 1), (dict(table=FAKE + 2), 4), (dict(lse=FAKE + 2), 4),
    (dict(o=0), 1), (dict(ws=0), 1), (dict(wsb=255), 1), (dict(n_pages=0), 2), (dict(new=-1), 2), (dict(len=-1), 2),
    (dict(T=(1 << 24) + 1), 3), (dict(T=1 << 15, n=1 << 15, page=1 << 16, pstride=1 << 24, max_pages=1 << 13, new=1), 3),
])
def test_forward_refuses(ralib, kw, status):
    assert _fwd(ralib.lib(), **kw) == status
    assert ralib.lib().ra_last_error().decode()


def test_empty_calls_launch_nothing(ralib):
    assert _fwd(ralib.lib(), T=0, q=0, o=0, ws=0) == 0
    assert _fwd(ralib.lib(), n=0, q=0, o=0, ws=0) == 0
    assert ralib.lib().ra_paged_append(0, 0, 0, 0, 0, 0, 0, 0, 4, 2, 128, 10, 16, 16 * 256, 4, 256, 0, 0, None) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(d=80), 3), (dict(Hkv=0), 2), (dict(page=20), 3), (dict(stride=255), 2), (dict(stride=260), 4), (dict(ps=4000), 2),
    (dict(k=0), 1), (dict(k=FAKE + 8), 4), (dict(wsb=16), 1), (dict(T=-1), 2), (dict(n_pages=0), 2), (dict(cu=0), 1),
])
def test_append_refuses(ralib, kw, status):
    a = dict(k=FAKE, T=8, n=2, Hkv=2, d=128, n_pages=10, page=16, ps=4096, max_pages=4, stride=256, cu=FAKE, wsb=256)
    a.update(kw)
    st = ralib.lib().ra_paged_append(a["k"], FAKE, FAKE, FAKE, FAKE, FAKE, a["cu"], a["T"], a["n"], a["Hkv"], a["d"],
                                     a["n_pages"], a["page"], a["ps"], a["max_pages"], a["stride"], FAKE, a["wsb"], None)
    assert st == status
    assert ralib.lib().ra_last_error().decode()


def test_workspace(ralib):
    f = ralib.ra_paged_attn_workspace_bytes
    assert f(64, 4, 8, 3, 128, 16, 300) == 0 and f(64, 4, 8, 2, 96, 16, 300) == 0
    for T, n, H, Hkv, d, new, length, W in ((1, 1, 32, 8, 128, 1, 131072, 0), (512, 1, 32, 8, 128, 512, 131072, 0),
                                            (4096, 300, 64, 8, 128, 2048, 1 << 20, 0), (64, 64, 16, 2, 64, 1, 1 << 17, 4096),
                                            (1, 1, 128, 1, 64, 1, 1 << 20, 0)):
        assert 256 <= f(T, n, H, Hkv, d, new, length, W, 4) <= 64 << 20
    big = (1 << 63) - 1
    assert f(100, 4, 8, 2, 128, big, 300) == f(100, 4, 8, 2, 128, 100, 300)
    assert 256 <= f(100, 4, 8, 2, 128, big, big, big, big) <= 64 << 20


def test_binding_refuses_host_tensors(ralib):
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    pages = torch.zeros((3, 16, 2, 64), dtype=torch.bfloat16)
    ints = torch.zeros((2, 4), dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        ralib.ra_paged_attn_fwd(x, pages, pages, ints, ints[:, 0].contiguous(), ints[0, :3].contiguous(), x, None, 4, 16,
                                workspace=ws)
    with pytest.raises(ValueError, match="CUDA"):
        ralib.ra_paged_append(x, x, pages, pages, ints, ints[:, 0].contiguous(), ints[0, :3].contiguous(), workspace=ws)
    with pytest.raises(ValueError, match="page must be contiguous"):
        ralib.ra_paged_append(x, x, pages.transpose(1, 2).contiguous().transpose(1, 2), pages, ints, ints, ints, workspace=ws)
