"""Calls from several host threads at once (tests/threads_probe.cpp), each with its own stream,
workspace and outputs.  A launch may not depend on what another thread's call set on the kernel in
between: calls that need very different amounts of shared memory all succeed and give what they
give alone."""
import ctypes
import os
import subprocess

import pytest
import torch

from conftest import ROOT
from synthetic_inputs import randn_bf16
from test_gpu_paged import Cache, cu_of

pytestmark = pytest.mark.gpu

THREADS, ROUNDS = 4, 4000


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("threads") / "threads_probe.so")
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-pthread", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "threads_probe.cpp"), "-o", out], check=True, capture_output=True)
    return ctypes.CDLL(out)


def ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def ptrs(ts):
    return (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])


def int64s(xs):
    return (ctypes.c_int64 * len(xs))(*xs)


def at_once(shape, H, T, sizes, ws_bytes, ralib, alone, run):
    """alone(i, o, lse): thread i's call through the binding; run(failed, o, lse, ws, stream): all threads."""
    want = [(torch.empty(shape, dtype=torch.bfloat16, device="cuda"), torch.empty((H, T), device="cuda")) for _ in sizes]
    for i, (o, lse) in enumerate(want):
        alone(i, o, lse)
    outs = [(torch.zeros_like(o), torch.zeros_like(lse)) for o, lse in want]
    ws = [ralib.new_workspace(ws_bytes) for _ in sizes]
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    failed = (ctypes.c_int * len(sizes))()
    run(failed, ptrs([o for o, _ in outs]), ptrs([lse for _, lse in outs]), ptrs(ws),
        (ctypes.c_void_p * len(sizes))(*[s.cuda_stream for s in streams]))
    torch.cuda.synchronize()
    assert list(failed) == [0] * len(sizes)
    for a, b in zip(outs, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# one kernel each: its warps share 16 rows, or take 16 rows each
@pytest.mark.parametrize("L,H,Hkv,windows", [(512, 2, 2, (20, 300)), (2000, 8, 8, (2, 60))])
@pytest.mark.parametrize("d", [64, 128])
def test_windowed_few_keys(ralib, gpu, probe, L, H, Hkv, windows, d):
    q, k, v = (randn_bf16((1, L, h, d), i).cuda() for i, h in enumerate((H, Hkv, Hkv)))
    sizes = windows * (THREADS // 2)

    def alone(i, o, lse):
        ralib.ra_window_attn_fwd(q, k, v, o, lse.view(1, H, L), 1, L, H, Hkv, d, sizes[i], workspace=ralib.new_workspace(256))

    def run(failed, o, lse, ws, streams):
        probe.ra_test_window_threads(
            ctypes.cast(ralib.lib().ra_window_attn_fwd, ctypes.c_void_p), THREADS, ROUNDS, failed, ptr(q), ptr(k), ptr(v),
            ctypes.c_int64(L), ctypes.c_int64(H), ctypes.c_int64(Hkv), d, int64s(sizes), o, lse, ws, streams)

    at_once((1, L, H, d), H, L, sizes, 256, ralib, alone, run)


@pytest.mark.parametrize("d,longest", [(64, 128), (128, 64)])
def test_paged_few_keys(ralib, gpu, probe, d, longest):
    H, Hkv, n_new, page = 8, 8, 40, 16
    c = Cache([n_new, n_new], page, Hkv, d, 3)
    c.fill_all()
    q, cu = randn_bf16((2 * n_new, H, d), 5).cuda(), cu_of([n_new, n_new])
    sizes = (1, longest) * (THREADS // 2)       # max_len: how many keys a block makes room for
    need = max(ralib.ra_paged_attn_workspace_bytes(2 * n_new, 2, H, Hkv, d, n_new, x) for x in sizes)

    def alone(i, o, lse):
        ralib.ra_paged_attn_fwd(q, c.k, c.v, c.table, c.seq_lens, cu, o, lse, n_new, sizes[i],
                                workspace=ralib.new_workspace(need))

    def run(failed, o, lse, ws, streams):
        n = ctypes.c_int64
        probe.ra_test_paged_threads(
            ctypes.cast(ralib.lib().ra_paged_attn_fwd, ctypes.c_void_p), THREADS, ROUNDS, failed, ptr(q), ptr(c.k),
            ptr(c.v), ptr(c.table), ptr(c.seq_lens), ptr(cu), n(2), n(n_new), n(H), n(Hkv), d, n(c.n_pages), n(page),
            n(c.max_pages), int64s(sizes), o, lse, ws, ctypes.c_size_t(need), streams)

    at_once((2 * n_new, H, d), H, 2 * n_new, sizes, need, ralib, alone, run)
