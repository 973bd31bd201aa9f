"""The tree attention's own units, runs, chains and chunks, counted on the host (tests/tree_probe.cu),
and what the calls on trees refuse."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import tree_reference as tr
from conftest import ROOT

CSRC = os.path.join(ROOT, "sequence_blockwise_softmax_gb300", "csrc")


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    out = str(tmp_path_factory.mktemp("tree") / "tree_probe.so")
    subprocess.run([nvcc, "-std=c++17", "-O2", "-shared", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"),
                    "-I", CSRC, os.path.join(ROOT, "tests", "tree_probe.cu"), "-o", out], check=True, capture_output=True)
    return ctypes.CDLL(out)


def _want(trees, lens, cap, T):
    want = np.zeros((T, cap), dtype=np.int32)

    def fill(window, sinks):
        t = 0
        for p, length in zip(trees, lens):
            for row in tr.sees(p, length - len(p), window, sinks):
                want[t, sorted(row)] = 1
                t += 1
        return want
    return fill


def _ints(x):
    return np.asarray(x, dtype=np.int32)


CASES = [
    # new tokens, lengths, page, max_pages, window, sinks
    ([1], [1], 16, 1, 0, 0),
    ([5, 1, 0, 32], [5, 300, 9, 1000], 16, 70, 0, 0),
    ([32, 20], [2000, 150], 64, 40, 3, 0),
    ([32, 20], [2000, 30], 64, 40, 7, 4),
    ([30, 17], [400, 17], 32, 20, 5, 40),          # sinks among the new tokens
    ([12, 32], [500, 600], 16, 40, 130, 20),
    ([9, 4], [3, 4], 16, 4, 0, 0),                 # more new tokens than length: negative places
    ([9, 4], [3, 4], 16, 4, 3, 2),
]
WIDE = CASES + [
    ([300, 1, 129], [300, 900, 2000], 128, 20, 0, 0),
    ([500], [3500], 16, 220, 9, 4),
    ([260, 140], [900, 3000], 64, 50, 200, 130),
    ([1024], [1500], 16, 100, 0, 0),
]


@pytest.mark.parametrize("shape", tr.SHAPES)
@pytest.mark.parametrize("new,lens,page,max_pages,window,sinks", WIDE)
def test_every_pair_once(probe, new, lens, page, max_pages, window, sinks, shape):
    trees = [tr.random_tree(n, shape, 7 + i) for i, n in enumerate(new)]
    T, cap = sum(new) + 2, max_pages * page
    want = _want(trees, lens, cap, T)(window, sinks)
    cu, sl = _ints(np.concatenate([[0], np.cumsum(new)])), _ints(lens)
    parents = _ints([x for t in trees for x in t] + [-9, 77])
    p = lambda a: ctypes.c_void_p(a.ctypes.data)
    # group, heads, tokens of a unit, lists, runs of each, places of a run at least, whether two Q tiles
    alone = ctypes.c_int(0)
    for group, heads, unit, streams, runs, least, two in ((1, 1, 256, 1, 1, 4, 1), (4, 3, 32, 3, 50, 4, 0), (5, 2, 25, 1, 7, 1, 0),
                                                          (128, 2, 1, 2, 76, 4, 0), (16, 8, 8, 8, 19, 2, 0),
                                                          (4, 4, 64, 2, 76, 2, 1), (1, 4, 512, 1, 60, 1, 1)):
        cnt = np.zeros((T, heads, cap), dtype=np.int32)
        assert probe.ra_test_tree_runs(p(sl), p(cu), p(parents), len(new), T, max_pages, page, group, heads, unit, max(new),
                                       window, sinks, streams, runs, least, two, ctypes.byref(alone), p(cnt)) == 0, (group, runs)
        assert np.array_equal(cnt, np.broadcast_to(want[:, None], cnt.shape)), (group, runs)
    assert alone.value > 0          # units were cut on their own in some of them
    if max(new) <= 32:
        for block in (max(new), 4, 1):
            cnt = np.zeros((T, cap), dtype=np.int32)
            assert probe.ra_test_tree_chunks(p(sl), p(cu), p(parents), len(new), T, max_pages, page, max(new), window, sinks,
                                             block, p(cnt)) == 0
            assert np.array_equal(cnt, want), block


@pytest.mark.parametrize("form", ["runs", "chunks"])
def test_what_is_no_tree_stays_inside(probe, form):
    """Parents of any value: a node out of its range counts as a root, nothing is read outside."""
    new, lens, page, max_pages = [8, 24], [60, 200], 16, 16
    r = np.random.RandomState(3)
    T, cap = sum(new), page * max_pages
    cu, sl = _ints([0, 8, 32]), _ints(lens)
    p = lambda a: ctypes.c_void_p(a.ctypes.data)
    for k in range(20):
        raw = r.choice([-2 ** 31, -7, -1, 0, 1, 5, 30, 32, 2 ** 31 - 1], T)
        raw = _ints(raw)
        trees = [[int(x) if -1 <= x < i else -1 for i, x in enumerate(raw[a:b])] for a, b in ((0, 8), (8, 32))]
        want = _want(trees, lens, cap, T)(0, 0)
        cnt = np.zeros((T, cap), dtype=np.int32)
        if form == "runs":
            rc = probe.ra_test_tree_runs(p(sl), p(cu), p(raw), 2, T, max_pages, page, 4, 1, 32, 24, 0, 0, 1, 3, 1, 0,
                                         ctypes.byref(ctypes.c_int(0)), p(cnt))
        else:
            rc = probe.ra_test_tree_chunks(p(sl), p(cu), p(raw), 2, T, max_pages, page, 24, 0, 0, 4, p(cnt))
        assert rc == 0 and np.array_equal(cnt, want)


FAKE = 0x10000      # 16-byte aligned, never dereferenced: every call below fails its checks first


def _tree(lib, **kw):
    a = dict(q=FAKE, kp=FAKE, par=FAKE, o=FAKE, lse=FAKE, T=64, n=4, H=8, Hkv=2, d=128, n_pages=10, page=16,
             pstride=16 * 2 * 128, max_pages=20, qs=1024, new=16, len=300, window=0, sinks=0, scale=0.0, flags=0, ws=FAKE,
             wsb=1 << 40)
    a.update(kw)
    return lib.ra_paged_tree_attn_fwd(a["q"], a["kp"], FAKE, FAKE, FAKE, FAKE, a["par"], a["o"], a["lse"], a["T"], a["n"],
                                      a["H"], a["Hkv"], a["d"], a["n_pages"], a["page"], a["pstride"], a["max_pages"],
                                      a["qs"], a["new"], a["len"], a["window"], a["sinks"], a["scale"], a["flags"], a["ws"],
                                      a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(new=1025), 3), (dict(par=0), 1), (dict(par=FAKE + 2), 4), (dict(d=96), 3), (dict(Hkv=3), 2), (dict(q=0), 1),
    (dict(o=FAKE + 8), 4), (dict(lse=FAKE + 2), 4), (dict(flags=8), 1), (dict(scale=float("nan")), 1), (dict(page=24), 3),
    (dict(page=8), 3), (dict(pstride=100), 2), (dict(qs=1000), 2), (dict(qs=1028), 4), (dict(window=-1), 1),
    (dict(sinks=-1), 1), (dict(wsb=256), 1), (dict(n_pages=0), 2), (dict(T=1 << 25), 3), (dict(max_pages=1 << 60), 3),
    (dict(new=-1), 2), (dict(qs=1 << 39), 3),
])
def test_tree_refuses(ralib, kw, status):
    assert _tree(ralib.lib(), **kw) == status
    assert ralib.lib().ra_last_error().decode()


def test_tree_workspace(ralib):
    w = ralib.ra_paged_tree_attn_workspace_bytes
    assert w(64, 4, 8, 2, 128, 16, 300) >= 256
    assert w(64, 4, 8, 2, 128, 1025, 3000) == 0 and w(64, 4, 8, 3, 128, 16, 300) == 0
    assert w(10000, 64, 32, 8, 128, 1024, 1 << 20) <= 64 << 20
    assert _tree(ralib.lib(), wsb=w(64, 4, 8, 2, 128, 16, 300) - 1) == 1


@pytest.mark.parametrize("kw", [dict(T=0), dict(n=0), dict(new=0)])
def test_nothing_to_do(ralib, kw):
    assert _tree(ralib.lib(), **dict(dict(q=0, kp=0, par=0, o=0, lse=0, ws=0), **kw)) == 0


def _rotary(lib, **kw):
    a = dict(q=FAKE, k=FAKE, qo=FAKE, kp=FAKE, par=0, freq=FAKE, T=8, n=2, H=8, Hkv=2, d=128, rot=128, n_pages=10, page=16,
             pstride=4096, max_pages=4, qs=1024, qos=1024, stride=256, flags=0, ws=FAKE, wsb=256)
    a.update(kw)
    return lib.ra_paged_append_rotary(a["q"], a["k"], FAKE, a["qo"], a["kp"], FAKE, FAKE, FAKE, FAKE, a["par"], a["freq"],
                                      a["T"], a["n"], a["H"], a["Hkv"], a["d"], a["rot"], a["n_pages"], a["page"],
                                      a["pstride"], a["max_pages"], a["qs"], a["qos"], a["stride"], a["flags"], a["ws"],
                                      a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rot=0), 3), (dict(rot=8), 3), (dict(rot=24), 3), (dict(rot=144), 3), (dict(d=64, rot=128), 3), (dict(rot=-16), 3),
    (dict(q=0), 1), (dict(qo=0), 1), (dict(k=0), 1), (dict(freq=0), 1), (dict(freq=FAKE + 2), 4), (dict(par=FAKE + 1), 4),
    (dict(q=FAKE + 8), 4), (dict(qs=1000), 2), (dict(qos=1000), 2), (dict(qos=1028), 4), (dict(stride=100), 2),
    (dict(stride=1 << 39), 3), (dict(qs=1 << 39), 3), (dict(flags=1), 1), (dict(wsb=128), 1), (dict(ws=0), 1), (dict(H=-1), 2),
    (dict(H=(1 << 16) + 1), 3), (dict(d=80), 3), (dict(page=20), 3), (dict(n_pages=0), 2), (dict(T=-1), 2),
])
def test_append_rotary_refuses(ralib, kw, status):
    assert _rotary(ralib.lib(), **kw) == status
    assert ralib.lib().ra_last_error().decode()


def test_append_rotary_in_place_keeps_the_stride(ralib):
    kw = dict(q=2 * FAKE, qo=2 * FAKE, wsb=128)
    assert _rotary(ralib.lib(), **kw) == 1 and "workspace" in ralib.lib().ra_last_error().decode()
    assert _rotary(ralib.lib(), qs=1280, **kw) == 1 and "in place" in ralib.lib().ra_last_error().decode()
    assert _rotary(ralib.lib(), qs=1280, T=1, **kw) == 1 and "workspace" in ralib.lib().ra_last_error().decode()


def test_append_rotary_nothing_to_do(ralib):
    for kw in (dict(T=0), dict(n=0)):
        assert _rotary(ralib.lib(), q=0, k=0, qo=0, kp=0, freq=0, ws=0, **kw) == 0


def _keep(lib, **kw):
    a = dict(kp=FAKE, par=FAKE, last=FAKE, lens=FAKE, new_lens=2 * FAKE, path=FAKE, T=8, n=2, layers=3, Hkv=2, d=128,
             n_pages=10, page=16, pstride=4096, lstride=40960, max_pages=4, ws=FAKE, wsb=256)
    a.update(kw)
    return lib.ra_paged_keep_path(a["kp"], FAKE, FAKE, a["lens"], FAKE, a["par"], a["last"], a["new_lens"], a["path"], a["T"],
                                  a["n"], a["layers"], a["Hkv"], a["d"], a["n_pages"], a["page"], a["pstride"], a["lstride"],
                                  a["max_pages"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(layers=-1), 2), (dict(layers=65537), 3), (dict(lstride=40952), 2), (dict(lstride=0), 2), (dict(lstride=40964), 4),
    (dict(lstride=-4096), 3), (dict(lstride=1 << 48), 3), (dict(lstride=4096, pstride=8192), 2), (dict(last=0), 1),
    (dict(par=0), 1), (dict(kp=0), 1), (dict(kp=FAKE + 8), 4), (dict(new_lens=0), 1), (dict(new_lens=FAKE), 1),
    (dict(path=FAKE + 2), 4), (dict(wsb=16), 1), (dict(d=32), 3), (dict(page=17), 3), (dict(n_pages=0), 2), (dict(n=-1), 2),
])
def test_keep_path_refuses(ralib, kw, status):
    assert _keep(ralib.lib(), **kw) == status
    assert ralib.lib().ra_last_error().decode()


def test_keep_path_nothing_to_do(ralib):
    assert _keep(ralib.lib(), n=0, kp=0, par=0, last=0, lens=0, new_lens=0, path=0, ws=0) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(layers=0, par=0), 1),                                             # a path is walked without layers too
    (dict(layers=0, n_pages=0), 2), (dict(layers=0, max_pages=0), 2),
    (dict(new_lens=3 * FAKE + 4), 1), (dict(new_lens=3 * FAKE - 4), 1),     # into last, seq_lens ..
    (dict(path=4 * FAKE), 1), (dict(path=4 * FAKE - 28), 1), (dict(path=4 * FAKE + 28), 1),    # .. parents ..
    (dict(path=2 * FAKE), 1), (dict(path=2 * FAKE + 4), 1),                 # .. the other output
])
def test_keep_path_outputs_apart(ralib, kw, status):
    """(the block table, cu_new and the values' pages are at FAKE)"""
    a = dict(lens=6 * FAKE, last=3 * FAKE, par=4 * FAKE, path=5 * FAKE)
    assert _keep(ralib.lib(), **dict(a, **kw)) == status
    assert _keep(ralib.lib(), **dict(a, wsb=16)) == 1 and "workspace" in ralib.lib().ra_last_error().decode()
