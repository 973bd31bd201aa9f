"""How often a weight is rounded: the mma.sync forms of the windowed and the paged forward keep P in
two bf16 parts, and the windowed backward rounds dS once and P not at all before it.

Forward, fp32 results.  P = hi + lo + r with hi = bf16(P), |P - hi| <= u P, and lo = bf16(P - hi),
so |r| <= u^2 P (u = 2^-8); O is divided by the sum of the unrounded P.  With EPS for every step
in 32 bits (window_reference.py), in the weights and in their sum:
    |O' - O| <= (u^2 + 2 EPS) (sum p |v| + |o|) + 1e-6.
Backward, fp32 gradients.  dS is rounded to bf16 once, from P and dP - D in 32 bits:
    |dQ' - dQ| <= sum ((u + EPS) |dS| + noise) |k| scale, and so dK with |q|;
the noise of D and dP as in window_reference.backward.  (u there and here is taken 1 % larger, for
the rounding of what has an error already.)

Each bound is one that a further rounding to bf16 would break: the same inputs, with P rounded once
(forward) or P rounded before dS is (backward), are beyond it in 64 bits.  Rows of one or two keys
show that best, since roundings of many keys cancel."""
import pytest
import torch

import window_reference as ref
from synthetic_inputs import randn_bf16
from test_gpu_paged import Cache, attend, cu_of, expect
from test_gpu_window import boundaries, inputs, reference, run_bwd, run_fwd

U = ref.U


def two_part_tolerance(p, v, o):
    spread = torch.einsum("bhlt,bthd->blhd", p, v.abs()) + o.abs()
    return (1.01 * U * U + 2 * ref.EPS) * spread + 1e-6


def rounded(p):
    """O's weights if P, relative to its row's largest, were one bf16 value."""
    top = p.amax(-1, keepdim=True).clamp_min(1e-30)
    return (p / top).bfloat16().double() * top


def check_forward(o, o_ref, p, v, what):
    tol = two_part_tolerance(p, v, o_ref)
    ref.assert_within(o, o_ref, tol, what)
    once = torch.einsum("bhlt,bthd->blhd", rounded(p), v)
    assert bool(((once - o_ref).abs() > tol).any()), what + ": the bound would pass P in one bf16 value"


@pytest.mark.gpu
@pytest.mark.parametrize("L,H,Hkv,d,window,sinks,cu", [
    # warps that share 16 rows: short windows, packed sequences, more keys
    (500, 2, 2, 64, 40, 4, None), (300, 4, 2, 128, 40, 3, [0, 1, 2, 4, 150, 300]), (400, 2, 1, 64, 300, 0, None),
    # warps with 16 rows each
    (2100, 16, 4, 128, 17, 3, None), (3000, 8, 8, 64, 30, 33, None), (4099, 4, 2, 128, 2, 0, None),
])
def test_windowed_forward(ralib, gpu, L, H, Hkv, d, window, sinks, cu):
    q, k, v, _ = inputs(1, L, H, Hkv, d, 3 * L + window)
    o, _ = run_fwd(ralib, q, k, v, window, sinks, boundaries(cu), torch.float32)
    _, _, _, vd, (o_ref, _, p) = reference(q, k, v, window, sinks, cu, d ** -0.5)
    check_forward(o, o_ref, p, vd, "O")


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens,H,Hkv,d,window,sinks", [
    ([1] * 8, [1, 2, 3, 2, 5, 9, 40, 100], 8, 2, 128, 0, 0),                   # clusters
    ([1, 2, 1, 3], [700, 2, 1500, 3], 8, 2, 64, 0, 0),
    ([1] * 200, [1 + i % 7 for i in range(200)], 8, 2, 64, 0, 0),             # a block to a pair
    ([1] * 120, [2 + i % 3 for i in range(118)] + [5000, 9000], 4, 2, 128, 0, 0),   # runs
    ([2, 1], [20000, 2], 8, 1, 128, 0, 0),                                   # pieces
    ([40, 3, 20], [40, 3, 50], 8, 8, 64, 0, 0),                              # few keys
    ([50, 45], [900, 45], 6, 2, 128, 3, 1),
])
def test_paged_forward(ralib, gpu, new, lens, H, Hkv, d, window, sinks):
    c = Cache(lens, 16, Hkv, d, sum(lens) + d)
    c.fill_all()
    q = randn_bf16((sum(new), H, d), 41).cuda()
    o, _, _ = attend(ralib, c, q, cu_of(new), new, torch.float32, window, sinks)
    t0, beyond = 0, False
    for s, n in enumerate(new):
        o_ref, _, p, vd = expect(c, q, new, s, t0, window, sinks)
        tol = two_part_tolerance(p, vd, o_ref)
        ref.assert_within(o[t0:t0 + n][None], o_ref, tol, "sequence %d" % s)
        beyond = beyond or bool(((torch.einsum("bhlt,bthd->blhd", rounded(p), vd) - o_ref).abs() > tol).any())
        t0 += n
    assert beyond, "the bound would pass P in one bf16 value"


def one_rounding(q, k, v, o, do, lse, ok, scale, Hkv, twice=False):
    """dQ, dK in 64 bits and their bounds with one rounding of dS; twice: dQ, dK with P rounded too."""
    B, L, H, d = q.shape
    s = (torch.einsum("blhd,bthd->bhlt", q, k) * scale).masked_fill(~ok, float("-inf"))
    p = torch.exp(s - lse[..., None])
    if twice:
        p = p.bfloat16().double()
    D = (do * o).sum(-1).transpose(1, 2)
    ds = p * (torch.einsum("blhd,bthd->bhlt", do, v) - D[..., None])
    if twice:
        ds = ds.bfloat16().double()
    noise = p * 2e-5 * (torch.einsum("blhd,bthd->bhlt", do.abs(), v.abs()) + (do * o).abs().sum(-1).transpose(1, 2)[..., None])
    off = (U * 1.01 + ref.EPS) * ds.abs() + noise
    shared = lambda x: x.reshape(B, L, Hkv, H // Hkv, d).sum(3)
    both = lambda w, a, b: (torch.einsum("bhlt,bthd->blhd", w, a) * scale, shared(torch.einsum("bhlt,blhd->bthd", w, b)) * scale)
    return both(ds, k, q), [x + 1e-6 for x in both(off, k.abs(), q.abs())]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L,H,Hkv,window,sinks,cu", [
    (1000, 4, 4, 2, 0, None), (900, 4, 4, 700, 0, [0] + list(range(1, 601, 3)) + [900]), (600, 4, 4, 1, 1, [0, 2, 4, 6, 300, 600]),
])
def test_windowed_backward(ralib, gpu, L, H, Hkv, window, sinks, cu, d):
    q, k, v, do = inputs(1, L, H, Hkv, d, 7 * L + d)
    cu_dev = boundaries(cu)
    o, lse = run_fwd(ralib, q, k, v, window, sinks, cu_dev, torch.float32)
    dq, dk, _ = run_bwd(ralib, q, k, v, o, do, lse, window, sinks, cu_dev, torch.float32)
    scale = d ** -0.5
    ok = ref.visible(L, window, sinks, cu, device="cuda")
    a = (q.double(), ref.expand_kv(k.double(), H), ref.expand_kv(v.double(), H), o.double(), do.double(), lse.double(), ok,
         scale, Hkv)
    grads, tols = one_rounding(*a)
    twice, _ = one_rounding(*a, twice=True)
    for name, x, g, t, w in zip(("dq", "dk"), (dq, dk), grads, tols, twice):
        ref.assert_within(x, g, t, name)
        assert bool(((w - g).abs() > t).any()), name + ": the bound would pass P rounded too"
