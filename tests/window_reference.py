"""Plain windowed attention and its gradients in 64 bits, and how far bf16 products may be off.

The tolerances count roundings, with u = 2^-8 the largest relative error of one rounding to
bf16, and take every other step (scores, exponentials, sums in 32 bits) as a relative error of
a weight of at most EPS: a score of d <= 128 products is summed in 32 bits with an error of at
most d 2^-23 sum|q k| scale, about 1e-4 at the inputs used here (sum|q k| scale <= 10), and the
exponential turns that into the same relative error of the weight.
"""
import torch

U = 2.0 ** -8
EPS = 2e-4


def visible(L, window, sinks, cu=None, device="cpu"):
    """[L, L] bool: query p sees key t."""
    p = torch.arange(L, device=device)
    start = torch.zeros(L, dtype=torch.long, device=device)
    if cu is not None:
        edges = torch.as_tensor(cu, dtype=torch.long, device=device)
        start = edges[torch.bucketize(p, edges, right=True) - 1]
    t = p[None, :]
    ok = (t <= p[:, None]) & (t >= start[:, None])
    return ok & ((t > p[:, None] - window) | (t < start[:, None] + sinks))


def expand_kv(x, H):
    return x.repeat_interleave(H // x.shape[2], 2)


def forward(q, k, v, ok, scale):
    """q [B, L, H, d] and k, v [B, T, H, d] (expanded) in 64 bits, ok [L, T] or [B, L, T].
    Returns O [B, L, H, d], LSE [B, H, L] and P [B, H, L, T]; a row that sees nothing gives 0 and -inf."""
    s = torch.einsum("blhd,bthd->bhlt", q, k) * scale
    s = s.masked_fill(~(ok if ok.dim() == 3 else ok[None])[:, None], float("-inf"))
    lse = torch.logsumexp(s, -1)
    safe = torch.where(torch.isneginf(lse), torch.zeros_like(lse), lse)
    p = torch.exp(s - safe[..., None])
    return torch.einsum("bhlt,bthd->blhd", p, v), lse, p


def forward_tolerance(p, v, o, out_bf16):
    """|O' - O| <= u/(1-u) sum p |v - O|: P is rounded to bf16 and O divided by the sum of the
    rounded P; with EPS for the weights and one more rounding of the result."""
    spread = torch.einsum("bhlt,bthd->blhd", p, v.abs()) + o.abs()
    return (U / (1 - U) + 2 * EPS) * spread + (U * 1.01 * o.abs() if out_bf16 else 0.0) + 1e-6


def backward(q, k, v, o, do, lse, ok, scale, Hkv):
    """The gradients from the forward's o and lse, and their tolerances: dV has one rounding per
    weight, dQ and dK two (P and dS); each with EPS, and the rounding of the result is the caller's."""
    B, L, H, d = q.shape
    s = torch.einsum("blhd,bthd->bhlt", q, k) * scale
    s = s.masked_fill(~ok, float("-inf"))
    p = torch.exp(s - lse[..., None])
    dp = torch.einsum("blhd,bthd->bhlt", do, v)
    dsum = (do * o).sum(-1).transpose(1, 2)
    ds = p * (dp - dsum[..., None])
    # D and dP are 32-bit sums of d terms
    noise = p * 2e-5 * (torch.einsum("blhd,bthd->bhlt", do.abs(), v.abs()) + (do * o).abs().sum(-1).transpose(1, 2)[..., None])
    ads = (2 * U * 1.01 + EPS) * ds.abs() + noise
    shared = lambda x: x.reshape(B, L, Hkv, H // Hkv, d).sum(3)   # a shared head's gradient
    dq = torch.einsum("bhlt,bthd->blhd", ds, k) * scale
    dk = shared(torch.einsum("bhlt,blhd->bthd", ds, q)) * scale
    dv = shared(torch.einsum("bhlt,blhd->bthd", p, do))
    tq = torch.einsum("bhlt,bthd->blhd", ads, k.abs()) * scale
    tk = shared(torch.einsum("bhlt,blhd->bthd", ads, q.abs())) * scale
    tv = shared(torch.einsum("bhlt,blhd->bthd", (U * 1.01 + EPS) * p, do.abs()))
    return (dq, dk, dv), (tq, tk, tv)


def assert_within(x, ref, tol, what):
    assert x.shape == ref.shape, what
    x = x.double()
    assert bool(torch.isfinite(x).all()), what + ": not finite"
    over = (x - ref).abs() - tol
    worst = over.max().item() if over.numel() else 0.0
    assert worst <= 0, "%s: off by %g where %g is allowed" % (
        what, (x - ref).abs().flatten()[over.argmax()].item(), tol.flatten()[over.argmax()].item())
