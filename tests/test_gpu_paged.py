"""Attention of new tokens over a paged cache, and appending to it, against the plain definition
in 64 bits.  Every place of the pool that no sequence holds is NaN."""
import random

import pytest
import torch

import window_reference as ref
from synthetic_inputs import randn_bf16

pytestmark = pytest.mark.gpu

NAN = float("nan")


class Cache:
    """Pools with pages in no order; interleaved: K and V of a page next to each other."""

    def __init__(self, lens, page, Hkv, d, seed, interleaved=False, spare=2, extra_cols=1):
        r = random.Random(seed)
        held = [-(-n // page) for n in lens]
        self.n_pages, self.page, self.Hkv, self.d, self.lens = sum(held) + spare, page, Hkv, d, lens
        ids = list(range(self.n_pages))
        r.shuffle(ids)
        self.max_pages = max(held + [1]) + extra_cols
        table = torch.full((len(lens), self.max_pages), -7, dtype=torch.int32)
        at = 0
        for s, h in enumerate(held):
            table[s, :h] = torch.tensor(ids[at:at + h], dtype=torch.int32)
            at += h
        self.rows = ids
        if interleaved:
            both = torch.full((self.n_pages, 2, page, Hkv, d), NAN, dtype=torch.bfloat16, device="cuda")
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = (torch.full((self.n_pages, page, Hkv, d), NAN, dtype=torch.bfloat16, device="cuda")
                              for _ in range(2))
        self.table = table.cuda()
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        # each sequence's keys and values, and their places in the pool
        self.ks = [randn_bf16((n, Hkv, d), seed + 2 * s + 1).cuda() for s, n in enumerate(lens)]
        self.vs = [randn_bf16((n, Hkv, d), seed + 2 * s + 2).cuda() for s, n in enumerate(lens)]

    def places(self, s, a, b):
        t = torch.arange(a, b, device="cuda")
        return self.table[s].long()[t // self.page], t % self.page

    def fill(self, s, a, b):
        if b > a:
            p, o = self.places(s, a, b)
            self.k[p, o], self.v[p, o] = self.ks[s][a:b], self.vs[s][a:b]

    def fill_all(self):
        for s, n in enumerate(self.lens):
            self.fill(s, 0, n)


def cu_of(new, first=0):
    return torch.tensor([first] + [first + sum(new[:i + 1]) for i in range(len(new))], dtype=torch.int32, device="cuda")


def attend(ra, c, q, cu, new, o_dtype, window=0, sinks=0, max_len=None, ws=None, check=True, lse=True):
    T, H, d = q.shape
    o = torch.full((T, H, d), NAN, dtype=o_dtype, device="cuda")
    lse = torch.full((H, T), NAN, dtype=torch.float32, device="cuda") if lse else None
    max_new, max_len = max(new), max(c.lens) if max_len is None else max_len
    if ws is None:
        ws = ra.new_workspace(ra.ra_paged_attn_workspace_bytes(T, len(new), H, c.Hkv, d, max_new, max_len, window, sinks))
    ra.ra_paged_attn_fwd(q, c.k, c.v, c.table, c.seq_lens, cu, o, lse, max_new, max_len, window, sinks, workspace=ws)
    if check:
        ra.ra_check_status(ws)
    return o, lse, ws


def expect(c, q, new, s, t0, window, sinks, scale=None):
    """O [n, H, d], LSE [H, n] and O's tolerance pieces (P, V) of sequence s's new tokens."""
    H, n, length = q.shape[1], new[s], c.lens[s]
    qd = q[t0:t0 + n].double()[None]
    kd, vd = (ref.expand_kv(x[s].double()[None], H) for x in (c.ks, c.vs))
    pos = torch.arange(length - n, length, device="cuda")[:, None]
    key = torch.arange(length, device="cuda")[None, :]
    ok = key <= pos
    if window:
        ok &= (key > pos - window) | (key < sinks)
    o, lse, p = ref.forward(qd, kd, vd, ok, q.shape[2] ** -0.5 if scale is None else scale)
    return o, lse, p, vd


def assert_paged(c, q, o, lse, new, window, sinks, first=0):
    t0 = first
    for s, n in enumerate(new):
        if n:
            oe, le, p, vd = expect(c, q, new, s, t0, window, sinks)
            tol = ref.forward_tolerance(p, vd, oe, o.dtype == torch.bfloat16)
            ref.assert_within(o[t0:t0 + n][None], oe, tol, "sequence %d O" % s)
            if lse is not None:
                ref.assert_within(lse[None, :, t0:t0 + n], le, torch.full_like(le, ref.EPS), "sequence %d LSE" % s)
        t0 += n


CASES = [
    # new, lens, H, Hkv, d, page, window, sinks
    ([1], [1], 4, 4, 64, 16, 0, 0),
    ([1], [2], 8, 1, 128, 16, 0, 0),
    ([1, 1, 1], [16, 17, 1000], 32, 8, 128, 16, 0, 0),
    ([1, 0, 1, 1], [129, 50, 4097, 128], 8, 8, 64, 32, 0, 0),
    ([1, 1], [5000, 20000], 16, 2, 64, 128, 700, 4),
    ([2, 3, 1, 4], [2, 700, 1300, 260], 10, 2, 128, 64, 0, 0),
    ([3], [9000], 24, 8, 128, 256, 100, 130),
    ([7, 1, 40], [7, 333, 2050], 12, 4, 64, 16, 0, 0),
    ([64, 65], [64, 1000], 4, 1, 128, 128, 0, 0),
    ([300, 1, 17], [300, 2500, 1040], 8, 2, 128, 32, 0, 0),
    ([257], [2257], 1, 1, 64, 512, 0, 0),
    ([200, 130], [3000, 130], 6, 2, 64, 16, 333, 5),
    ([5, 6], [1500, 40], 66, 2, 128, 16, 0, 0),
    ([2], [900], 128, 1, 64, 64, 0, 0),
    ([33], [12000], 8, 1, 128, 16, 0, 0),
    ([40], [9000], 60, 60, 64, 64, 0, 0),      # long parts and a short one
    ([200], [7000], 60, 30, 128, 16, 0, 0),
    # few keys: short prompts, short windows
    ([40, 3, 64, 0, 1], [40, 60, 64, 9, 1], 8, 8, 128, 16, 0, 0),
    ([90, 1, 128], [90, 128, 128], 6, 2, 64, 32, 0, 0),
    ([100, 40], [3000, 900], 20, 4, 64, 16, 20, 4),
    ([70, 33], [1500, 33], 3, 1, 128, 64, 7, 17),
    ([35, 41], [50, 41], 64, 1, 64, 128, 0, 0),
]


@pytest.mark.parametrize("new,lens,H,Hkv,d,page,window,sinks", CASES)
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_paged_matches_definition(ralib, gpu, new, lens, H, Hkv, d, page, window, sinks, o_dtype):
    c = Cache(lens, page, Hkv, d, sum(lens) + H)
    c.fill_all()
    q = randn_bf16((sum(new), H, d), 99 + H).cuda()
    o, lse, _ = attend(ralib, c, q, cu_of(new), new, o_dtype, window, sinks)
    assert_paged(c, q, o, lse, new, window, sinks)


@pytest.mark.parametrize("max_len", [1, 1 << 20])
@pytest.mark.parametrize("n", [1, 9, 40])
def test_any_guess_of_the_length(ralib, gpu, n, max_len):
    """max_len only guides the split: far too short or too long, the results hold."""
    new, lens = [n, n], [6000, 77]
    c = Cache(lens, 32, 2, 128, 5)
    c.fill_all()
    q = randn_bf16((sum(new), 8, 128), 4).cuda()
    o, lse, _ = attend(ralib, c, q, cu_of(new), new, torch.bfloat16, max_len=max_len)
    assert_paged(c, q, o, lse, new, 0, 0)


@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("d", [64, 128])
def test_strided_tensors(ralib, gpu, n, d):
    """q as the first part of a fused projection; K and V of a page in one block."""
    new, lens, H, Hkv = [n, n, n], [400, n, 2000], 8, 2
    c = Cache(lens, 16, Hkv, d, 6, interleaved=True)
    c.fill_all()
    fused = randn_bf16((sum(new), H + 2 * Hkv, d), 8).cuda()
    q = fused[:, :H]
    o, lse, _ = attend(ralib, c, q, cu_of(new), new, torch.bfloat16)
    assert_paged(c, q, o, lse, new, 0, 0)


@pytest.mark.parametrize("n", [1, 50])
def test_rows_outside_the_sequences_are_left(ralib, gpu, n):
    """Padded rows of q, NaN, before the first and behind the last sequence: neither read into a
    result nor written."""
    new, lens, H, Hkv, d = [n, n], [300, 900], 8, 2, 128
    c = Cache(lens, 16, Hkv, d, 7)
    c.fill_all()
    q = torch.full((3 + 2 * n + 9, H, d), NAN, dtype=torch.bfloat16, device="cuda")
    q[3:3 + 2 * n] = randn_bf16((2 * n, H, d), 9).cuda()
    o, lse, _ = attend(ralib, c, q, cu_of(new, 3), new, torch.bfloat16)
    assert_paged(c, q, o, lse, new, 0, 0, first=3)
    for x in (o[:3], o[3 + 2 * n:], lse[:, :3], lse[:, 3 + 2 * n:]):
        assert bool(torch.isnan(x).all())


@pytest.mark.parametrize("n", [1, 30])
def test_without_lse(ralib, gpu, n):
    new, lens = [n], [3000]
    c = Cache(lens, 64, 1, 64, 3)
    c.fill_all()
    q = randn_bf16((n, 4, 64), 2).cuda()
    o, _, _ = attend(ralib, c, q, cu_of(new), new, torch.bfloat16, lse=False)
    assert_paged(c, q, o, None, new, 0, 0)


@pytest.mark.parametrize("n", [1, 40])
def test_window_does_not_read_freed_pages(ralib, gpu, n):
    """Pages between the sinks and the window are given back: their entries are -1."""
    window, sinks, page, length = 300, 4, 32, 5000
    new = [n]
    c = Cache([length], page, 2, 128, 12)
    c.fill_all()
    gone = torch.arange(1, (length - n - window) // page)
    c.table[0, gone] = -1
    q = randn_bf16((n, 8, 128), 3).cuda()
    o, lse, _ = attend(ralib, c, q, cu_of(new), new, torch.bfloat16, window, sinks)
    assert_paged(c, q, o, lse, new, window, sinks)


@pytest.mark.parametrize("n", [1, 40])
def test_bad_tables_are_reported(ralib, gpu, n):
    """A page outside the pool, more new tokens than announced or than the sequence has, a length
    past the table's row: reported, nothing out of range, and the next call is fine."""
    new, lens, H, d = [n, n], [500, 800], 8, 128
    c = Cache(lens, 16, 2, d, 13, extra_cols=0)
    c.fill_all()
    q = randn_bf16((2 * n, H, d), 3).cuda()
    good = c.table.clone()
    ws = attend(ralib, c, q, cu_of(new), new, torch.bfloat16)[2]
    for bad in (-1, c.n_pages, 2 ** 31 - 1):
        c.table[1, 3] = bad
        attend(ralib, c, q, cu_of(new), new, torch.bfloat16, ws=ws, check=False)
        with pytest.raises(ralib.RAError, match="page"):
            ralib.ra_check_status(ws)
        c.table.copy_(good)
    for length in (0, 10 ** 6, -3):
        c.seq_lens[0] = length
        o, lse, _ = attend(ralib, c, q, cu_of(new), new, torch.bfloat16, ws=ws, check=False)
        with pytest.raises(ralib.RAError, match="lengths"):
            ralib.ra_check_status(ws)
        if length <= 0:      # every position is negative or the token's own
            assert bool((o[:n - 1] == 0).all()) and bool(torch.isneginf(lse[:, :n - 1]).all())
    c.seq_lens.copy_(torch.tensor(lens))
    if n > 1:
        attend(ralib, c, q, cu_of(new), [n - 3], torch.bfloat16, ws=ws, check=False)
        with pytest.raises(ralib.RAError, match="lengths"):
            ralib.ra_check_status(ws)
    o, lse, _ = attend(ralib, c, q, cu_of(new), new, torch.bfloat16, ws=ws)
    assert_paged(c, q, o, lse, new, 0, 0)


@pytest.mark.parametrize("n", [1, 25])
def test_scores_far_from_zero(ralib, gpu, n):
    """Keys whose scores lie far from the others', in one part of the split or another."""
    new, lens, H, d = [n], [9000], 8, 128
    c = Cache(lens, 64, 1, d, 17)
    q = randn_bf16((n, H, d), 3).cuda()
    q[..., 0] = 16.0
    c.ks[0][..., 0] = -30.0
    c.ks[0][1000:1004, :, 0] = 25.0
    c.ks[0][8000, :, 0] = 27.0
    c.fill_all()
    o, lse, _ = attend(ralib, c, q, cu_of(new), new, torch.float32)
    oe, le, p, vd = expect(c, q, new, 0, 0, 0, 0)
    # a score's 32-bit sum here is as large as 16 * 30 and off by up to 2e-4 more
    ref.assert_within(o[None], oe, 2 * ref.forward_tolerance(p, vd, oe, False), "O")
    ref.assert_within(lse[None], le, 1e-5 * le.abs() + 4 * ref.EPS, "LSE")


@pytest.mark.parametrize("n_first", [30, 300])
def test_append_attend_replayed(ralib, gpu, n_first):
    """A prompt and then single tokens, as a server runs them: append and attend captured once and
    replayed while lengths, tables and tokens change; every step's rows are the definition's, and
    a second run gives the same bits."""
    H, Hkv, d, page, n = 8, 2, 128, 16, 3
    lens = [n_first + 20, n_first + 3, 2 * n_first]
    c = Cache(lens, page, Hkv, d, 23)
    q = [randn_bf16((x, H, d), 50 + s).cuda() for s, x in enumerate(lens)]
    ws = ralib.new_workspace(64 << 20)
    first = [x - 8 for x in lens]
    # the prompt in one call, tokens strided
    kv = torch.cat([torch.stack([c.ks[s][:first[s]], c.vs[s][:first[s]]], 1) for s in range(n)])
    c.seq_lens.copy_(torch.tensor(first))
    ralib.ra_paged_append(kv[:, 0], kv[:, 1], c.k, c.v, c.table, c.seq_lens, cu_of(first), workspace=ws)
    kq, vq, qq = (torch.empty((n, h, d), dtype=torch.bfloat16, device="cuda") for h in (Hkv, Hkv, H))
    o, lse = torch.empty_like(qq), torch.empty((H, n), device="cuda")
    cu = cu_of([1] * n)

    def step():
        ralib.ra_paged_append(kq, vq, c.k, c.v, c.table, c.seq_lens, cu, workspace=ws)
        ralib.ra_paged_attn_fwd(qq, c.k, c.v, c.table, c.seq_lens, cu, o, lse, 1, max(lens), workspace=ws)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    full = c.lens
    with torch.cuda.graph(graph):
        step()
    for i in range(8):
        now = [x + i + 1 for x in first]
        c.seq_lens.copy_(torch.tensor(now))
        for s in range(n):
            kq[s], vq[s], qq[s] = c.ks[s][now[s] - 1], c.vs[s][now[s] - 1], q[s][now[s] - 1]
        graph.replay()
        once = o.clone(), lse.clone()
        step()
        assert torch.equal(o, once[0]) and torch.equal(lse, once[1])
        c.lens = now
        keep = c.ks, c.vs
        c.ks, c.vs = [x[:m] for x, m in zip(c.ks, now)], [x[:m] for x, m in zip(c.vs, now)]
        assert_paged(c, qq, o, lse, [1] * n, 0, 0)
        c.ks, c.vs = keep
    ralib.ra_check_status(ws)
    c.lens = full
    for s in range(n):      # the pool holds the tokens, and nothing else was written
        p, at = c.places(s, 0, full[s])
        assert torch.equal(c.k[p, at], c.ks[s]) and torch.equal(c.v[p, at], c.vs[s])
    written = sum(full)
    assert int((~torch.isnan(c.k[..., 0, 0])).sum()) == written


@pytest.mark.parametrize("Hkv,d,page", [(1, 64, 16), (3, 64, 32), (8, 128, 256)])
def test_append(ralib, gpu, Hkv, d, page):
    """Tokens of ragged sequences land at their places only; rows outside the sequences stay out."""
    new, lens = [5, 0, 700, 1], [5, 33, 1000, 4 * page]
    c = Cache(lens, page, Hkv, d, 31)
    T = 2 + sum(new) + 4
    kn, vn = randn_bf16((T, Hkv, d), 1).cuda(), randn_bf16((T, Hkv, d), 2).cuda()
    ws = ralib.new_workspace(256)
    ralib.ra_paged_append(kn, vn, c.k, c.v, c.table, c.seq_lens, cu_of(new, 2), workspace=ws)
    ralib.ra_check_status(ws)
    k, v = (torch.full((c.n_pages, page, Hkv, d), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    t = 2
    for s, m in enumerate(new):
        p, at = c.places(s, lens[s] - m, lens[s])
        k[p, at], v[p, at] = kn[t:t + m], vn[t:t + m]
        t += m
    assert torch.equal(k.view(torch.int16), c.k.view(torch.int16))
    assert torch.equal(v.view(torch.int16), c.v.view(torch.int16))


def test_append_reports_bad_places(ralib, gpu):
    c = Cache([100, 200], 16, 2, 64, 37)
    kn = randn_bf16((2, 2, 64), 1).cuda()
    ws = ralib.new_workspace(256)
    cu = cu_of([1, 1])
    for entry, length in ((-1, 200), (c.n_pages, 200), (0, 0), (0, 10 ** 6)):
        c.table[1, 199 // 16] = entry
        c.seq_lens[1] = length
        before = c.k.clone()
        ralib.ra_paged_append(kn, kn, c.k, c.v, c.table, c.seq_lens, cu, workspace=ws)
        with pytest.raises(ralib.RAError, match="page"):
            ralib.ra_check_status(ws)
        p, at = c.places(0, 99, 100)
        before[p, at] = kn[:1]
        assert torch.equal(before.view(torch.int16), c.k.view(torch.int16))


def test_binding_refuses(ralib, gpu):
    c = Cache([100], 16, 2, 64, 37)
    q = randn_bf16((1, 4, 64), 1).cuda()
    o, cu, ws = torch.empty_like(q), cu_of([1]), ralib.new_workspace(256)

    def call(**kw):
        a = dict(q=q, k=c.k, v=c.v, table=c.table, lens=c.seq_lens, cu=cu, o=o, ws=ws)
        a.update(kw)
        ralib.ra_paged_attn_fwd(a["q"], a["k"], a["v"], a["table"], a["lens"], a["cu"], a["o"], None, 1, 100,
                                workspace=a["ws"])

    for kw in (dict(q=q.half()), dict(k=c.k.float()), dict(table=c.table.long()), dict(o=o.half())):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(lens=c.seq_lens.repeat(2)), dict(cu=cu[:1]), dict(v=c.v[:1]), dict(o=o[:, :2]), dict(ws=None),
               dict(q=q[..., :32]), dict(table=c.table.cpu()), dict(k=c.k.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ralib.RAError):
        call(q=randn_bf16((1, 3, 64), 1).cuda(), o=torch.empty((1, 3, 64), dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("new_max", [1, 90])
def test_more_units_than_multiprocessors(ralib, gpu, new_max):
    """Many ragged sequences: several units follow one another on each multiprocessor."""
    r = random.Random(new_max)
    new = [r.randint(1, new_max) for _ in range(70)]
    lens = [x + r.randint(0, 3000) for x in new]
    c = Cache(lens, 64, 8, 128, 71)
    c.fill_all()
    q = randn_bf16((sum(new), 32, 128), 5).cuda()
    o, lse, _ = attend(ralib, c, q, cu_of(new), new, torch.bfloat16)
    assert_paged(c, q, o, lse, new, 0, 0)


@pytest.mark.parametrize("n,longest", [(300, 60), (300, 2500), (40, 900)])
def test_many_sequences(ralib, gpu, n, longest):
    """More sequences than a block has threads, some without new tokens; short ones, a CTA each."""
    r = random.Random(n + longest)
    new = [r.randint(0, 1) for _ in range(n)]
    lens = [x + r.randint(0, longest) for x in new]
    c = Cache(lens, 16, 8, 64, 73)
    c.fill_all()
    q = randn_bf16((sum(new), 16, 64), 5).cuda()
    o, lse, _ = attend(ralib, c, q, cu_of(new), new, torch.bfloat16)
    assert_paged(c, q, o, lse, new, 0, 0)


def test_workspace_left_by_other_calls(ralib, gpu):
    """A workspace that other calls have written to, its header apart, serves the split forms."""
    c = Cache([20000, 5000], 64, 2, 128, 79)
    c.fill_all()
    ws = ralib.new_workspace(64 << 20)
    for n in (1, 40, 1):
        ws[256:] = torch.randint(0, 256, (ws.numel() - 256,), dtype=torch.uint8, device="cuda")
        q = randn_bf16((2 * n, 8, 128), 4 + n).cuda()
        for _ in range(3):
            o, lse, _ = attend(ralib, c, q, cu_of([n, n]), [n, n], torch.bfloat16, ws=ws)
            assert_paged(c, q, o, lse, [n, n], 0, 0)


@pytest.mark.parametrize("new,lens,H,Hkv,d,window,sinks", [
    # clusters of 2, 4, 8 and 16: few keys, single tokens and several, no new tokens, windows
    ([1, 1], [1, 100], 8, 8, 128, 0, 0),
    ([1, 0, 2] * 20, [5, 0, 128] * 20, 8, 2, 64, 0, 0),
    ([1] * 70, [16 * i + 1 for i in range(44, 9, -1)] * 2, 4, 1, 128, 0, 0),
    ([1, 3], [200, 250], 16, 2, 128, 0, 0),
    ([2, 1, 0, 1], [700, 2000, 3, 1], 32, 8, 64, 0, 0),
    ([1] * 12, [90 * i + 300 for i in range(12)], 16, 2, 128, 300, 4),
    ([4, 8], [3000, 17], 8, 2, 128, 0, 0),
    ([1], [8192], 32, 8, 128, 0, 0),
    ([2], [8000], 16, 1, 64, 0, 0),
    ([1, 2], [6000, 9000], 16, 2, 64, 4000, 130),
    ([16], [5000], 2, 2, 128, 0, 0),
    # pieces of two row tiles, and runs of a third as many pairs as CTAs
    ([4, 8], [9500, 12000], 8, 2, 128, 0, 0),
    ([1] * 16, [7000 + 16 * i for i in range(16)], 16, 8, 64, 0, 0),
])
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_clusters(ralib, gpu, new, lens, H, Hkv, d, window, sinks, o_dtype):
    c = Cache(lens, 32, Hkv, d, sum(lens))
    c.fill_all()
    T = sum(new) + 3                # rows behind the last sequence are left alone
    q = randn_bf16((T, H, d), 31).cuda()
    ws = ralib.new_workspace(ralib.ra_paged_attn_workspace_bytes(T, len(new), H, Hkv, d, max(new), max(lens), window, sinks))
    first = None
    for _ in range(3):
        o, lse, _ = attend(ralib, c, q, cu_of(new), new, o_dtype, window, sinks, ws=ws)
        assert_paged(c, q, o, lse, new, window, sinks)
        assert bool(torch.isnan(o[sum(new):]).all()) and bool(torch.isnan(lse[:, sum(new):]).all())
        assert first is None or torch.equal(first, o[:sum(new)])
        first = o[:sum(new)]


def test_counters_are_never_floats(ralib, gpu):
    """The words a split call counts in are signalling NaNs in their upper half,
    so that no float that arithmetic left in a workspace can pass for one, and
    an own one for each call."""
    c = Cache([20000, 5000], 64, 2, 128, 80)
    c.fill_all()
    q = randn_bf16((2, 8, 128), 6).cuda()
    tags = []
    for _ in range(2):
        ws = ralib.new_workspace(64 << 20)
        o, lse, _ = attend(ralib, c, q, cu_of([1, 1]), [1, 1], torch.bfloat16, ws=ws)
        assert_paged(c, q, o, lse, [1, 1], 0, 0)
        words = {w & (1 << 64) - 1 for w in ws[256:256 + 4096].view(torch.int64).tolist()} - {0}
        assert len(words) == 1
        tags += words
    assert tags[0] != tags[1] and all(w >> 52 == 0xffa and w & 1023 == 0 for w in tags)


@pytest.mark.parametrize("new,longest,H,Hkv,d", [
    ([1] * 300, 900, 16, 8, 64),            # a CTA for each pair, more of them than counters
    ([1] * 70, 3000, 16, 8, 64),            # equal runs of all pairs
    ([1, 1], 9000, 8, 1, 128),              # a cluster for each pair
    ([1, 1], 20000, 8, 1, 128),             # pieces of one pair
    ([4, 8], 3000, 8, 2, 128),              # two row tiles
    ([40], 20000, 8, 2, 128),               # tiles, split and joined
    ([40, 2, 300], 700, 8, 2, 64),
    ([40, 2, 60], 100, 8, 2, 64),           # few keys
])
def test_workspace_is_not_left(ralib, gpu, new, longest, H, Hkv, d):
    """Nothing is written past the bytes a call asks for."""
    r = random.Random(longest)
    lens = [longest] + [max(x, r.randint(1, longest)) for x in new[1:]]
    c = Cache(lens, 16, Hkv, d, 91)
    c.fill_all()
    q = randn_bf16((sum(new), H, d), 4).cuda()
    need = ralib.ra_paged_attn_workspace_bytes(sum(new), len(new), H, Hkv, d, max(new), longest)
    room = torch.zeros(need + (1 << 20), dtype=torch.uint8, device="cuda")
    room[need:] = 0xA5
    o, lse, _ = attend(ralib, c, q, cu_of(new), new, torch.bfloat16, ws=room[:need])
    assert bool((room[need:] == 0xA5).all())
    assert_paged(c, q, o, lse, new, 0, 0)


@pytest.mark.parametrize("n,length,window", [(1, 3000, 0), (40, 3000, 0), (40, 50, 0), (9, 3000, 20)])
def test_pool_past_32_bits(ralib, gpu, n, length, window):
    """Pages whose offsets pass 2^32 elements and 2^33 bytes, in each form; appended and read."""
    Hkv, d, page, H = 8, 128, 256, 16
    n_pages = (1 << 32) // (page * Hkv * d) + 40
    c = Cache([length], page, Hkv, d, 5)
    pool = torch.empty((n_pages, 2, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
    held = -(-length // page)
    high = torch.randperm(30)[:held] + n_pages - 35
    c.n_pages, c.k, c.v = n_pages, pool[:, 0], pool[:, 1]
    c.table = torch.full((1, held + 1), -1, dtype=torch.int32, device="cuda")
    c.table[0, :held] = high.to(torch.int32).cuda()
    pool[n_pages - 40:] = NAN
    c.fill(0, 0, length - n)
    ws = ralib.new_workspace(64 << 20)
    ralib.ra_paged_append(c.ks[0][length - n:], c.vs[0][length - n:], c.k, c.v, c.table, c.seq_lens, cu_of([n]), workspace=ws)
    q = randn_bf16((n, H, d), 3).cuda()
    o, lse, _ = attend(ralib, c, q, cu_of([n]), [n], torch.bfloat16, window, 4 if window else 0, ws=ws)
    assert_paged(c, q, o, lse, [n], window, 4 if window else 0)


def test_two_streams_two_workspaces(ralib, gpu):
    """The same call on two streams at once, a workspace each, many times over."""
    c = Cache([20000, 300, 7000], 64, 2, 128, 83)
    c.fill_all()
    new = [1, 1, 1]
    q = randn_bf16((3, 8, 128), 4).cuda()
    want, want_lse, _ = attend(ralib, c, q, cu_of(new), new, torch.bfloat16)
    cu = cu_of(new)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.empty_like(want), torch.empty_like(want_lse), ralib.new_workspace(16 << 20)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (o, lse, ws) in zip(streams, outs):
            ralib.ra_paged_attn_fwd(q, c.k, c.v, c.table, c.seq_lens, cu, o, lse, 1, max(c.lens), workspace=ws, stream=s)
    torch.cuda.synchronize()
    for o, lse, _ in outs:
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
