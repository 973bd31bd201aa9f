"""Sliding-window attention with sinks on the GPU, forward and backward, against the plain
definition in 64 bits (tests/window_reference.py)."""
import pytest
import torch

import window_reference as ref
from synthetic_inputs import randn_bf16

pytestmark = pytest.mark.gpu

# B, L, H, Hkv, d, window, sinks, boundaries
CASES = [
    (1, 1, 1, 1, 64, 1, 0, None),
    (2, 1, 2, 1, 128, 7, 3, None),
    (1, 127, 2, 2, 128, 1, 0, None),
    (1, 128, 2, 2, 64, 128, 4, None),
    (1, 129, 4, 2, 128, 2, 200, None),
    (2, 700, 4, 1, 64, 100, 4, None),
    (1, 700, 6, 2, 128, 129, 130, None),
    (1, 513, 3, 3, 64, 256, 1, None),
    (1, 700, 2, 2, 128, 5000, 9, None),
    (1, 900, 4, 4, 128, 33, 150, [0, 128, 256, 400, 900]),
    (1, 701, 4, 2, 64, 50, 4, [0, 1, 1, 300, 301, 650, 701]),
    (1, 2300, 2, 1, 128, 60, 5, None),
    (1, 2600, 2, 2, 64, 77, 131, [0, 30, 2048, 2049, 2060, 2600]),
    (1, 800, 2, 2, 128, 40, 6, [0, 300, 500]),
    # tokens behind the last sequence, in each form
    (1, 800, 4, 2, 64, 500, 6, [0, 300, 641]),
    (1, 1200, 4, 2, 128, 300, 140, [0, 5, 1025]),
    (1, 1500, 2, 1, 128, 260, 0, [0, 1024]),
    (1, 400, 2, 2, 64, 5, 3, [0, 0]),
    (1, 900, 2, 2, 64, 700, 3, [0, 0, 1]),
    # the form with few keys at one wave of blocks above, at several here (the first two pack sequences)
    (1, 2100, 16, 4, 128, 17, 3, [0, 1, 40, 41, 300, 1000, 2049, 2100]),
    (1, 2090, 8, 8, 64, 30, 33, [0, 70, 1024, 2000]),
    (2, 2050, 8, 2, 64, 60, 4, None),
    (1, 4099, 4, 2, 128, 1, 0, None),
    (1, 2049, 12, 4, 128, 2, 65, None),
    # and the tensor-core form on short and ragged inputs
    (1, 300, 2, 1, 128, 260, 3, [0, 290, 300]),
    (2, 257, 2, 2, 64, 257, 0, None),
    (1, 1025, 8, 1, 128, 300, 200, [0, 5, 700, 1025]),
    (1, 3000, 8, 8, 128, 129, 4, None),
]


def inputs(B, L, H, Hkv, d, seed, tokens=None):
    """q, k, v, dO; what lies behind the first `tokens` tokens is NaN."""
    xs = [randn_bf16((B, L, h, d), seed + i).cuda() for i, h in enumerate((H, Hkv, Hkv, H))]
    for x in xs:
        x[:, L if tokens is None else tokens:] = float("nan")
    return xs


def boundaries(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")


def run_fwd(ra, q, k, v, window, sinks, cu, o_dtype, scale=0.0):
    B, L, H, d = q.shape
    o = torch.full(q.shape, float("nan"), dtype=o_dtype, device="cuda")
    lse = torch.full((B, H, L), float("nan"), dtype=torch.float32, device="cuda")
    ws = ra.new_workspace(256)
    ra.ra_window_attn_fwd(q, k, v, o, lse, B, L, H, k.shape[2], d, window, sinks, scale=scale, cu_seqlens=cu,
                          workspace=ws)
    ra.ra_check_status(ws)
    return o, lse


def run_bwd(ra, q, k, v, o, do, lse, window, sinks, cu, g_dtype, scale=0.0):
    B, L, H, d = q.shape
    Hkv = k.shape[2]
    grads = [torch.full(x.shape, float("nan"), dtype=g_dtype, device="cuda") for x in (q, k, v)]
    n = 0 if cu is None else cu.numel() - 1
    ws = ra.new_workspace(ra.ra_window_attn_bwd_workspace_bytes(B, L, H, Hkv, d, window, sinks, n))
    ra.ra_window_attn_bwd(q, k, v, o, do, lse, *grads, B, L, H, Hkv, d, window, sinks, scale=scale, cu_seqlens=cu,
                          workspace=ws)
    ra.ra_check_status(ws)
    return grads


def reference(q, k, v, window, sinks, cu, scale):
    H = q.shape[2]
    ok = ref.visible(q.shape[1], window, sinks, cu, device="cuda")
    qd, kd, vd = q.double(), ref.expand_kv(k.double(), H), ref.expand_kv(v.double(), H)
    return ok, qd, kd, vd, ref.forward(qd, kd, vd, ok, scale)


@pytest.mark.parametrize("B,L,H,Hkv,d,window,sinks,cu", CASES)
@pytest.mark.parametrize("o_dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_window_matches_definition(ralib, gpu, B, L, H, Hkv, d, window, sinks, cu, o_dtype):
    n = L if cu is None else cu[-1]           # tokens in sequences; the others' rows stay as they were
    q, k, v, do = inputs(B, L, H, Hkv, d, 7 * L + window, n)
    cu_dev = boundaries(cu)
    scale = d ** -0.5
    o, lse = run_fwd(ralib, q, k, v, window, sinks, cu_dev, o_dtype)
    assert bool(torch.isnan(o[:, n:]).all()) and bool(torch.isnan(lse[:, :, n:]).all())
    ok, qd, kd, vd, (o_ref, lse_ref, p) = reference(*(x[:, :n] for x in (q, k, v)), window, sinks, cu, scale)
    what = "window %d sinks %d" % (window, sinks)
    ref.assert_within(o[:, :n], o_ref, ref.forward_tolerance(p, vd, o_ref, o_dtype == torch.bfloat16), what + " O")
    ref.assert_within(lse[:, :, :n], lse_ref, torch.full_like(lse_ref, ref.EPS), what + " LSE")
    del p
    grads, tols = ref.backward(qd, kd, vd, o[:, :n].double(), do[:, :n].double(), lse[:, :, :n].double(), ok, scale, Hkv)
    for g_dtype in (torch.float32, torch.bfloat16):
        out = run_bwd(ralib, q, k, v, o, do, lse, window, sinks, cu_dev, g_dtype)
        for name, x, g, t in zip(("dq", "dk", "dv"), out, grads, tols):
            end = ref.U * 1.01 * g.abs() if g_dtype == torch.bfloat16 else 0.0
            ref.assert_within(x[:, :n], g, t + end + 1e-5, what + " " + name)
            assert bool(torch.isnan(x[:, n:]).all()), what + " " + name + " behind the sequences"


def test_scores_far_from_zero(ralib, gpu):
    """Rows whose exponentials leave the range of a fixed reference: large scores in the sinks,
    in the window or in neither, so that the reference moves while part of a tile is masked."""
    B, L, H, d, window, sinks = 1, 600, 2, 128, 100, 4
    q, k, v, _ = inputs(B, L, H, H, d, 5)
    q, k = q.float(), k.float()
    q[..., 0] = 16.0
    k[..., 0] = -30.0
    k[:, :2, :, 0] = 30.0
    k[:, 300:310, :, 0] = 28.0
    q, k = q.bfloat16(), k.bfloat16()
    o, lse = run_fwd(ralib, q, k, v, window, sinks, None, torch.float32)
    _, _, _, vd, (o_ref, lse_ref, p) = reference(q, k, v, window, sinks, None, d ** -0.5)
    # a score's 32-bit sum here is as large as 16 * 30 and off by up to 2e-4 more
    ref.assert_within(o, o_ref, 2 * ref.forward_tolerance(p, vd, o_ref, False), "O")
    ref.assert_within(lse, lse_ref, 1e-5 * lse_ref.abs() + 4 * ref.EPS, "LSE")


@pytest.mark.parametrize("d", [64, 128])
def test_a_window_of_everything_is_the_ring_call(ralib, gpu, d):
    """Without a window the result is ra_ring_attn_fwd's causal sweep over one shard, bit for bit."""
    B, L, H = 2, 700, 2
    q, k, v, _ = inputs(B, L, H, H, d, 11)
    o, lse = run_fwd(ralib, q, k, v, L, 5, None, torch.float32)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    ws = ralib.new_workspace(256)
    ralib.ra_ring_attn_fwd(q, k, v, o2, lse2, B, L, H, d, 1, "contiguous", True, flags=ralib.RA_FLAG_SEQ_ORDER,
                           workspace=ws)
    ralib.ra_check_status(ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_gradients_repeat_and_replay(ralib, gpu):
    """Forward and backward in one graph, replayed on changed inputs, give what separate calls give,
    bit for bit, with the sinks' partial sums in the same workspace."""
    B, L, H, Hkv, d, window, sinks = 1, 4500, 4, 2, 64, 300, 130
    q, k, v, do = inputs(B, L, H, Hkv, d, 21)
    ws = ralib.new_workspace(ralib.ra_window_attn_bwd_workspace_bytes(B, L, H, Hkv, d, window, sinks))
    o, lse = torch.empty_like(q), torch.empty((B, H, L), dtype=torch.float32, device="cuda")
    grads = [torch.empty_like(x) for x in (q, k, v)]

    def step():
        ralib.ra_window_attn_fwd(q, k, v, o, lse, B, L, H, Hkv, d, window, sinks, workspace=ws)
        ralib.ra_window_attn_bwd(q, k, v, o, do, lse, *grads, B, L, H, Hkv, d, window, sinks, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (31, 41):
        for x, y in zip((q, k, v, do), inputs(B, L, H, Hkv, d, seed)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        replayed = [x.clone() for x in (o, lse, *grads)]
        for x in (o, lse, *grads):
            x.zero_()
        step()
        for a, b in zip(replayed, (o, lse, *grads)):
            assert torch.equal(a, b)
    ralib.ra_check_status(ws)


@pytest.mark.parametrize("L,sinks,cu", [(700, 5, None), (3000, 131, [0, 10, 1500, 2900]), (600, 0, None)])
def test_workspace_is_not_left(ralib, gpu, L, sinks, cu):
    """The backward writes nothing past the bytes it asks for."""
    H, Hkv, d, window = 4, 2, 64, 50
    q, k, v, do = inputs(1, L, H, Hkv, d, 17)
    cu_dev = boundaries(cu)
    o, lse = run_fwd(ralib, q, k, v, window, sinks, cu_dev, torch.bfloat16)
    want = run_bwd(ralib, q, k, v, o, do, lse, window, sinks, cu_dev, torch.bfloat16)
    need = ralib.ra_window_attn_bwd_workspace_bytes(1, L, H, Hkv, d, window, sinks, 0 if cu is None else len(cu) - 1)
    room = torch.zeros(need + (1 << 20), dtype=torch.uint8, device="cuda")
    room[need:] = 0xA5
    grads = [torch.empty_like(x) for x in (q, k, v)]
    ralib.ra_window_attn_bwd(q, k, v, o, do, lse, *grads, 1, L, H, Hkv, d, window, sinks, cu_seqlens=cu_dev,
                             workspace=room[:need])
    assert bool((room[need:] == 0xA5).all())
    n = L if cu is None else cu[-1]
    for x, y in zip(grads, want):
        assert torch.equal(x[:, :n], y[:, :n])


def test_side_stream(ralib, gpu):
    B, L, H, d = 1, 1000, 2, 128
    q, k, v, _ = inputs(B, L, H, H, d, 3)
    want = run_fwd(ralib, q, k, v, 64, 2, None, torch.bfloat16)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse, ws = torch.empty_like(q), torch.empty((B, H, L), device="cuda"), ralib.new_workspace(256)
    side.wait_stream(torch.cuda.current_stream())
    ralib.ra_window_attn_fwd(q, k, v, o, lse, B, L, H, H, d, 64, 2, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(o, want)


def test_binding_refuses(ralib, gpu):
    B, L, H, d = 1, 64, 2, 64
    q, k, v, _ = inputs(B, L, H, H, d, 3)
    o, lse, ws = torch.empty_like(q), torch.empty((B, H, L), device="cuda"), ralib.new_workspace(256)
    call = lambda **kw: ralib.ra_window_attn_fwd(*[kw.get(n, x) for n, x in (("q", q), ("k", k), ("v", v), ("o", o),
                                                                              ("lse", lse))],
                                                 B, L, H, H, d, kw.get("window", 8), 0, workspace=kw.get("ws", ws))
    call()
    with pytest.raises(TypeError):
        call(q=q.half())
    with pytest.raises(ValueError):
        call(k=k[:, :32])
    with pytest.raises(ValueError):
        call(v=v.transpose(1, 2))
    with pytest.raises(ValueError):
        call(o=o.cpu())
    with pytest.raises(TypeError):
        call(lse=lse.double())
    with pytest.raises(ralib.RAError):
        call(window=0)
    with pytest.raises(ValueError):
        call(ws=None)
