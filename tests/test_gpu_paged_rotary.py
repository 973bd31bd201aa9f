"""Appending to a paged cache with the position rotation applied on the way, against the definition in
64 bits."""
import math
import random

import pytest
import torch

import tree_reference as tr
from synthetic_inputs import randn_bf16
from test_gpu_paged import NAN, Cache, cu_of

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
# The angle is off by 9e-8 at position 2^29 (64-bit floating point) and 9e-8 where it goes to fp32, the cosine
# and sine by 2^-23 and less, and the two products and their sum by three roundings to fp32: relative to |x| + |y|.
ANGLE = 6e-7


def frequencies(half, base=10000.0):
    return (base ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()


def rotated(x, pos, freq, pairs):
    """x [T, heads, d] turned in 64 bits, and its tolerance."""
    rot, y = 2 * freq.numel(), x.double()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if pairs else (y[..., :rot // 2], y[..., rot // 2:rot])
    # a position below 2^29 times an fp32 frequency is exact in 64 bits
    phi = (pos.double()[:, None] * freq.double())[:, None]
    ra, rb = a * phi.cos() - b * phi.sin(), a * phi.sin() + b * phi.cos()
    out, tol = y.clone(), torch.zeros_like(y)
    for dst, new in ((out, (ra, rb)), (tol, [U * n.abs() + (1 + U) * ANGLE * (a.abs() + b.abs()) for n in (ra, rb)])):
        if pairs:
            dst[..., 0:rot:2], dst[..., 1:rot:2] = new
        else:
            dst[..., :rot // 2], dst[..., rot // 2:rot] = new
    return out, tol


def places(c, new, trees=None):
    """Each new token's page and offset there, and its position."""
    page, off, pos = [], [], []
    for s, n in enumerate(new):
        before = c.lens[s] - n
        p, o = c.places(s, before, c.lens[s])
        page.append(p)
        off.append(o)
        pos += [before + (i if trees is None else len(tr.path(trees[s], i)) - 1) for i in range(n)]
    return torch.cat(page), torch.cat(off), torch.tensor(pos, dtype=torch.int64, device="cuda")


def check(ra, c, new, H, rot, pairs, trees=None, first=0, tail=0, in_place=False, freq=None, seed=1):
    T, Hkv, d = first + sum(new) + tail, c.Hkv, c.d
    qkv = torch.full((T, H + 2 * Hkv, d), NAN, dtype=torch.bfloat16, device="cuda")
    qkv[first:T - tail] = randn_bf16((sum(new), H + 2 * Hkv, d), seed).cuda()
    was = qkv.clone()
    q, kn, vn = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    out = q if in_place else torch.full((T, H, d), NAN, dtype=torch.bfloat16, device="cuda")
    freq = frequencies(rot // 2) if freq is None else freq
    parents = None if trees is None else torch.tensor([7] * first + [x for t in trees for x in t] + [-9] * tail,
                                                      dtype=torch.int32, device="cuda")
    before = c.k.clone(), c.v.clone()
    ws = ra.new_workspace(256)
    ra.ra_paged_append_rotary(q if H else None, kn, vn, out if H else None, c.k, c.v, c.table, c.seq_lens, cu_of(new, first), freq,
                              parents=parents, pairs=pairs, workspace=ws)
    ra.ra_check_status(ws)
    page, off, pos = places(c, new, trees)
    rows = slice(first, T - tail)
    src = was[rows]
    ke, kt = rotated(src[:, H:H + Hkv], pos, freq, pairs)
    over = ((c.k[page, off].double() - ke).abs() - kt).max().item() if sum(new) else 0
    assert over <= 0, "keys: %g" % over
    assert torch.equal(c.v[page, off], src[:, H + Hkv:])
    if H:
        qe, qt = rotated(src[:, :H], pos, freq, pairs)
        over = ((out[rows].double() - qe).abs() - qt).max().item() if sum(new) else 0
        assert over <= 0, "queries: %g" % over
        assert bool(torch.isnan(out[:first]).all()) and bool(torch.isnan(out[T - tail:]).all())
        assert torch.equal(out[rows][..., rot:], src[:, :H][..., rot:])
    # nothing else was written
    for now, then in ((c.k, before[0]), (c.v, before[1])):
        now = now.clone()
        now[page, off] = then[page, off]
        assert torch.equal(now.view(torch.int16), then.view(torch.int16))


CASES = [
    # new, lens, H, Hkv, d, page, rot, pairs
    ([1], [1], 4, 4, 64, 16, 64, False),
    ([1], [1], 1, 1, 128, 16, 128, True),
    ([1] * 64, [17 * i + 1 for i in range(64)], 32, 8, 128, 16, 128, False),
    ([5, 0, 700, 1], [5, 33, 1000, 64], 3, 1, 64, 16, 16, False),
    ([5, 0, 700, 1], [5, 33, 1000, 64], 6, 2, 128, 64, 96, True),
    ([0, 0, 3, 0], [4, 0, 900, 17], 5, 5, 128, 256, 48, False),
    ([2000, 1500], [2000, 4000], 32, 8, 128, 64, 128, False),
    ([333], [500], 0, 3, 128, 32, 32, True),                     # no queries
    ([1] * 400, [i + 1 for i in range(400)], 2, 1, 64, 16, 32, False),
    ([100], [100], 128, 1, 64, 128, 64, True),
    ([3000], [3000], 1, 1, 64, 16, 64, False),                   # few items a token
]


@pytest.mark.parametrize("new,lens,H,Hkv,d,page,rot,pairs", CASES)
@pytest.mark.parametrize("in_place", [False, True])
def test_append_rotary(ralib, gpu, new, lens, H, Hkv, d, page, rot, pairs, in_place):
    c = Cache(lens, page, Hkv, d, 31)
    check(ralib, c, new, H, rot, pairs, first=2, tail=3, in_place=in_place and H > 0)


@pytest.mark.parametrize("shape", tr.SHAPES)
@pytest.mark.parametrize("new,lens", [([26, 0, 60, 1], [3000, 4, 60, 2]), ([1024, 7], [1200, 9])])
def test_trees(ralib, gpu, new, lens, shape):
    c = Cache(lens, 32, 2, 64, 33)
    check(ralib, c, new, 4, 32, shape == "bush", trees=[tr.random_tree(n, shape, 5) for n in new], first=1, tail=1)


@pytest.mark.parametrize("empty", [40, 200])
def test_many_empty_sequences(ralib, gpu, empty):
    """Tokens of neighbouring rows whose sequences lie far apart in number."""
    new = [2] + [0] * empty + [1] + [0] * empty + [40] + [0] * 5
    c = Cache([n + 3 for n in new], 16, 1, 64, 34)
    check(ralib, c, new, 2, 64, False, first=1)


def test_far_positions(ralib, gpu):
    """Positions up to 2^29 - 1: the angle is right to 1e-7 of a radian, whatever the turns before it."""
    page, d, rot = 65536, 128, 128
    lens = [1 << 29, (1 << 28) + 12345, 131072]
    c = Cache([40, 40, 40], 64, 1, d, 35)          # (its tables are replaced)
    c.page, c.n_pages, c.max_pages, c.lens = page, 3, 8192, lens
    c.k, c.v = (torch.full((3, page, 1, d), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c.table = torch.full((3, 8192), -1, dtype=torch.int32, device="cuda")
    for s, n in enumerate(lens):
        c.table[s, (n - 1) // page] = 2 - s
    c.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    check(ralib, c, [20, 20, 20], 2, rot, False)


@pytest.mark.parametrize("freq", [[0.0] * 8, [1.0] * 8, [-0.3] * 8, [7.5, 1000.0, 3.1415927, 6.2831855, 1e-30, -4.0, 0.5, 2.0]])
def test_any_frequency(ralib, gpu, freq):
    c = Cache([300], 16, 1, 64, 36)
    check(ralib, c, [100], 2, 16, False, freq=torch.tensor(freq, device="cuda"))


def test_position_zero_is_a_copy(ralib, gpu):
    c = Cache([1], 16, 2, 128, 38)
    k = randn_bf16((1, 2, 128), 3).cuda()
    ws = ralib.new_workspace(256)
    ralib.ra_paged_append_rotary(None, k, k, None, c.k, c.v, c.table, c.seq_lens, cu_of([1]), frequencies(64), workspace=ws)
    p, at = c.places(0, 0, 1)
    assert torch.equal(c.k[p, at], k) and torch.equal(c.v[p, at], k)


def test_bad_places_are_reported(ralib, gpu):
    """A page outside the pool, a place outside the table, more tokens than the length, no tree: reported;
    the others' keys and every sequence's queries are right."""
    c = Cache([100, 200], 16, 2, 64, 37)
    kn, q = randn_bf16((2, 2, 64), 1).cuda(), randn_bf16((2, 4, 64), 2).cuda()
    out, ws, cu, freq = torch.empty_like(q), ralib.new_workspace(256), cu_of([1, 1]), frequencies(32)

    def call(parents=None):
        ralib.ra_paged_append_rotary(q, kn, kn, out, c.k, c.v, c.table, c.seq_lens, cu, freq, parents=parents, workspace=ws)
        with pytest.raises(ralib.RAError, match="page"):
            ralib.ra_check_status(ws)

    good = c.table.clone()
    for entry, length in ((-1, 200), (c.n_pages, 200), (0, 0), (0, 10 ** 6)):
        c.table[1, 199 // 16], c.seq_lens[1] = entry, length
        before = c.k.clone()
        call()
        p, at = c.places(0, 99, 100)
        pos = torch.tensor([99, length - 1], device="cuda")
        ke, kt = rotated(kn[:1], pos[:1], freq, False)
        assert bool(((c.k[p, at].double() - ke).abs() <= kt).all())
        qe, qt = rotated(q, pos, freq, False)
        assert bool(((out.double() - qe).abs() <= qt).all())
        before[p, at] = c.k[p, at]
        assert torch.equal(before.view(torch.int16), c.k.view(torch.int16))
    c.table.copy_(good)
    c.seq_lens[1] = 200
    for bad in (0, -2, 2 ** 31 - 1):
        call(torch.tensor([-1, bad], dtype=torch.int32, device="cuda"))
    ralib.ra_paged_append_rotary(q, kn, kn, out, c.k, c.v, c.table, c.seq_lens, cu, freq, workspace=ws)
    ralib.ra_check_status(ws)


def test_more_tokens_than_a_tree_holds(ralib, gpu):
    """The first 1024 nodes are taken, the rows behind them left out and reported."""
    c = Cache([1100], 64, 1, 64, 39)
    kn, q = randn_bf16((1100, 1, 64), 1).cuda(), randn_bf16((1100, 2, 64), 2).cuda()
    out = torch.full_like(q, NAN)
    ws = ralib.new_workspace(256)
    parents = torch.arange(-1, 1099, dtype=torch.int32, device="cuda")
    ralib.ra_paged_append_rotary(q, kn, kn, out, c.k, c.v, c.table, c.seq_lens, cu_of([1100]), frequencies(32), parents=parents,
                                 workspace=ws)
    with pytest.raises(ralib.RAError):
        ralib.ra_check_status(ws)
    assert bool(torch.isfinite(out[:1024]).all()) and bool(torch.isnan(out[1024:]).all())
    p, at = c.places(0, 0, 1100)
    assert bool(torch.isfinite(c.v[p, at][:1024]).all()) and bool(torch.isnan(c.v[p, at][1024:]).all())


def test_pool_past_32_bits(ralib, gpu):
    Hkv, d, page = 8, 128, 256
    n_pages = (1 << 32) // (page * Hkv * d) + 40
    c = Cache([600], page, Hkv, d, 5)
    pool = torch.empty((n_pages, 2, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
    kn, vn = randn_bf16((600, Hkv, d), 1).cuda(), randn_bf16((600, Hkv, d), 2).cuda()
    c.table[0, :3] = torch.tensor([n_pages - 3, n_pages - 30, n_pages - 11], dtype=torch.int32)
    freq = frequencies(64)
    ws = ralib.new_workspace(256)
    ralib.ra_paged_append_rotary(None, kn, vn, None, pool[:, 0], pool[:, 1], c.table, c.seq_lens, cu_of([600]), freq, workspace=ws)
    ralib.ra_check_status(ws)
    p, at = c.places(0, 0, 600)
    ke, kt = rotated(kn, torch.arange(600, device="cuda"), freq, False)
    assert bool(((pool[p, 0, at].double() - ke).abs() <= kt).all()) and torch.equal(pool[p, 1, at], vn)


def test_binding_refuses(ralib, gpu):
    c = Cache([100], 16, 2, 64, 37)
    k, q = randn_bf16((1, 2, 64), 1).cuda(), randn_bf16((1, 4, 64), 1).cuda()
    freq, cu, ws = frequencies(32), cu_of([1]), ralib.new_workspace(256)
    par = torch.tensor([-1], dtype=torch.int32, device="cuda")

    def call(**kw):
        a = dict(q=q, k=k, v=k, out=q, freq=freq, par=par, ws=ws)
        a.update(kw)
        ralib.ra_paged_append_rotary(a["q"], a["k"], a["v"], a["out"], c.k, c.v, c.table, c.seq_lens, cu, a["freq"],
                                     parents=a["par"], workspace=a["ws"])

    for kw in (dict(q=q.float()), dict(k=k.half()), dict(freq=freq.double()), dict(par=par.long()), dict(freq=None)):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(out=None), dict(q=None), dict(v=k[:, :1]), dict(out=q[:, :2]), dict(freq=freq.cpu()), dict(freq=freq[None]),
               dict(par=par.repeat(2)), dict(ws=None), dict(q=q[..., :32], out=q[..., :32])):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(freq=freq[:4]), dict(freq=freq[:0])):
        with pytest.raises(ralib.RAError):
            call(**kw)
