"""Rows all of whose scores lie far below zero, past the exponents of 32 bits (2^-128), or far
above and below it: the first keys a row sees must not be scaled by what its empty sum was.

Keys lie near one direction u per head (k = s (u + 0.1 n)) and queries near -u, so that every
score is about -s^2 |u|^2 scale = -200.  A score's 32-bit sum of d products is then off by at most
d 2^-23 200 (3.1e-3 at d = 128), the bound every comparison here uses for a weight's relative
error and for LSE.
"""
import pytest
import torch

import oracle
import window_reference as ref
from conftest import assert_attention_close
from test_gpu_attention import run_ring
from test_gpu_paged import Cache, assert_paged, attend, cu_of
from test_gpu_window import reference, run_bwd, run_fwd

pytestmark = pytest.mark.gpu

SCORE = 200.0


def near(shape, sign, seed):
    """bf16 [..., heads, d] rows near sign * s * u, u the same for all heads."""
    g = torch.Generator().manual_seed(seed)
    d = shape[-1]
    u = torch.randn((d,), generator=torch.Generator().manual_seed(d))
    s = (SCORE / (u.square().sum().item() * d ** -0.5)) ** 0.5
    return (sign * s * (u + 0.1 * torch.randn(shape, generator=g))).bfloat16()


@pytest.fixture
def far(monkeypatch):
    monkeypatch.setattr(ref, "EPS", 128 * 2.0 ** -23 * SCORE)


@pytest.mark.parametrize("d,window,sinks", [(64, 20, 4), (128, 20, 4), (64, 400, 4), (128, 400, 4), (128, 900, 0)])
def test_window(ralib, gpu, far, d, window, sinks):
    B, L, H, Hkv = 1, 900, 4, 2
    q, k = near((B, L, H, d), -1, 1).cuda(), near((B, L, Hkv, d), 1, 2).cuda()
    v, do = (torch.randn((B, L, h, d), generator=torch.Generator().manual_seed(h)).bfloat16().cuda() for h in (Hkv, H))
    o, lse = run_fwd(ralib, q, k, v, window, sinks, None, torch.float32)
    scale = d ** -0.5
    ok, qd, kd, vd, (o_ref, lse_ref, p) = reference(q, k, v, window, sinks, None, scale)
    assert lse_ref.max() < -120
    ref.assert_within(o, o_ref, ref.forward_tolerance(p, vd, o_ref, False), "O")
    ref.assert_within(lse, lse_ref, torch.full_like(lse_ref, ref.EPS), "LSE")
    grads, tols = ref.backward(qd, kd, vd, o.double(), do.double(), lse.double(), ok, scale, Hkv)
    for x, g, t in zip(run_bwd(ralib, q, k, v, o, do, lse, window, sinks, None, torch.float32), grads, tols):
        ref.assert_within(x, g, t + 1e-5, "gradient")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,lens", [([1, 2], [600, 5000]), ([40, 33], [40, 60]), ([300, 50], [900, 4000]),
                                      ([100], [12000])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 5)])
def test_paged(ralib, gpu, far, d, new, lens, window, sinks):
    H, Hkv = 4, 2
    c = Cache(lens, 32, Hkv, d, 3)
    c.ks = [near((n, Hkv, d), 1, 10 + s).cuda() for s, n in enumerate(lens)]
    c.fill_all()
    q = near((sum(new), H, d), -1, 4).cuda()
    o, lse, _ = attend(ralib, c, q, cu_of(new), new, torch.float32, window, sinks)
    assert_paged(c, q, o, lse, new, window, sinks)


@pytest.mark.parametrize("layout,causal,d", [("striped", True, 128), ("zigzag", True, 64), ("contiguous", False, 128)])
def test_ring(ralib, gpu, layout, causal, d):
    B, L, H, N = 1, 1024, 2, 4
    q, k = near((B, L, H, d), -1, 5), near((B, L, H, d), 1, 6)
    v = torch.randn((B, L, H, d), generator=torch.Generator().manual_seed(7)).bfloat16()
    o_ref, lse_ref = oracle.full_attention(q, k, v, causal=causal)
    assert lse_ref.max() < -120
    for flags in (0, 1):
        o, lse = run_ring(ralib, q, k, v, N, layout, causal, flags=flags)
        assert_attention_close(o, o_ref, lse, lse_ref, layout)


@pytest.mark.parametrize("d,window,sinks", [(64, 20, 4), (128, 20, 4), (64, 400, 200), (128, 400, 200), (128, 900, 0)])
def test_window_both_signs(ralib, gpu, far, d, window, sinks):
    """Scores of +200 and -200 in runs of keys: a row's reference moves up and, past the sinks, stays."""
    B, L, H, Hkv = 1, 900, 4, 2
    q, k = near((B, L, H, d), -1, 1).cuda(), near((B, L, Hkv, d), 1, 2).cuda()
    for a, b in ((0, 3), (130, 170), (420, 650)):
        k[:, a:b] = -k[:, a:b]
    v, do = (torch.randn((B, L, h, d), generator=torch.Generator().manual_seed(h)).bfloat16().cuda() for h in (Hkv, H))
    o, lse = run_fwd(ralib, q, k, v, window, sinks, None, torch.float32)
    scale = d ** -0.5
    ok, qd, kd, vd, (o_ref, lse_ref, p) = reference(q, k, v, window, sinks, None, scale)
    assert lse_ref.max() > 120
    ref.assert_within(o, o_ref, ref.forward_tolerance(p, vd, o_ref, False), "O")
    ref.assert_within(lse, lse_ref, torch.full_like(lse_ref, ref.EPS), "LSE")
    grads, tols = ref.backward(qd, kd, vd, o.double(), do.double(), lse.double(), ok, scale, Hkv)
    for x, g, t in zip(run_bwd(ralib, q, k, v, o, do, lse, window, sinks, None, torch.float32), grads, tols):
        ref.assert_within(x, g, t + 1e-5, "gradient")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,lens", [([1, 2], [600, 5000]), ([40, 33], [40, 60]), ([300, 50], [900, 4000]),
                                      ([100], [12000])])
def test_paged_both_signs(ralib, gpu, far, d, new, lens):
    H, Hkv = 4, 2
    c = Cache(lens, 32, Hkv, d, 3)
    c.ks = [near((n, Hkv, d), 1, 10 + s).cuda() for s, n in enumerate(lens)]
    for x in c.ks:
        x[17:33] = -x[17:33]
        x[len(x) // 2:len(x) // 2 + 5] = -x[len(x) // 2:len(x) // 2 + 5]
    c.fill_all()
    q = near((sum(new), H, d), -1, 4).cuda()
    o, lse, _ = attend(ralib, c, q, cu_of(new), new, torch.float32)
    assert_paged(c, q, o, lse, new, 0, 0)
