"""Attention of trees of new tokens over a paged cache against the plain definition in 64 bits.
Every place of the pool that no sequence holds is NaN."""
import random

import pytest
import torch

import tree_reference as tr
import window_reference as ref
from synthetic_inputs import randn_bf16
from test_gpu_paged import NAN, Cache, cu_of

pytestmark = pytest.mark.gpu


def trees_of(new, shape, seed=3):
    return [tr.random_tree(n, shape, seed + i) for i, n in enumerate(new)]


def flat(trees, first=0, tail=0):
    return torch.tensor([-5] * first + [x for t in trees for x in t] + [99] * tail, dtype=torch.int32, device="cuda")


def attend(ra, c, q, cu, trees, o_dtype, window=0, sinks=0, max_len=None, ws=None, check=True, lse=True, first=0, parents=None):
    T, H, d = q.shape
    o = torch.full((T, H, d), NAN, dtype=o_dtype, device="cuda")
    lse = torch.full((H, T), NAN, dtype=torch.float32, device="cuda") if lse else None
    max_new, max_len = max(len(t) for t in trees), max(c.lens) if max_len is None else max_len
    if ws is None:
        ws = ra.new_workspace(ra.ra_paged_tree_attn_workspace_bytes(T, len(trees), H, c.Hkv, d, max_new, max_len, window, sinks))
    if parents is None:
        parents = flat(trees, first, T - first - sum(len(t) for t in trees))
    ra.ra_paged_tree_attn_fwd(q, c.k, c.v, c.table, c.seq_lens, cu, parents, o, lse, max_new, max_len, window, sinks, workspace=ws)
    if check:
        ra.ra_check_status(ws)
    return o, lse, ws


def expect(c, q, tree, s, t0, window, sinks, scale=None):
    H, n, length = q.shape[1], len(tree), c.lens[s]
    qd = q[t0:t0 + n].double()[None]
    kd, vd = (ref.expand_kv(x[s].double()[None], H) for x in (c.ks, c.vs))
    ok = torch.zeros((n, length), dtype=torch.bool)
    for i, places in enumerate(tr.sees(tree, length - n, window, sinks)):
        ok[i, sorted(places)] = True
    o, lse, p = ref.forward(qd, kd, vd, ok.cuda(), q.shape[2] ** -0.5 if scale is None else scale)
    return o, lse, p, vd


def assert_trees(c, q, o, lse, trees, window, sinks, first=0):
    t0 = first
    for s, tree in enumerate(trees):
        n = len(tree)
        if n:
            oe, le, p, vd = expect(c, q, tree, s, t0, window, sinks)
            tol = ref.forward_tolerance(p, vd, oe, o.dtype == torch.bfloat16)
            ref.assert_within(o[t0:t0 + n][None], oe, tol, "sequence %d O" % s)
            if lse is not None:
                ref.assert_within(lse[None, :, t0:t0 + n], le, torch.full_like(le, ref.EPS), "sequence %d LSE" % s)
        t0 += n


CASES = [
    # new, lens, H, Hkv, d, page, window, sinks
    ([1], [1], 4, 4, 64, 16, 0, 0),                             # a root over nothing
    ([8], [8], 8, 2, 128, 16, 0, 0),
    ([8], [1000], 32, 8, 128, 16, 0, 0),                        # few rows: a cluster to a pair
    ([4, 0, 7, 8], [1290, 50, 4097, 128], 16, 4, 64, 32, 0, 0),
    ([32, 20, 1], [20000, 33, 700], 2, 2, 128, 64, 0, 0),       # a cluster each, 32 nodes
    ([16] * 30, [300 + 90 * i for i in range(30)], 8, 8, 64, 16, 0, 0),
    ([3, 4, 2], [9000, 30000, 200], 16, 2, 128, 128, 700, 4),
    ([30, 17], [400, 17], 1, 1, 64, 32, 5, 40),                 # sinks among the new tokens
    ([32, 9], [600, 2000], 4, 4, 128, 16, 3, 2),                # a window shorter than the tree is deep
    ([26, 1, 60], [700, 333, 2050], 12, 4, 64, 16, 0, 0),       # many rows: tiles
    ([60], [8192], 32, 8, 128, 64, 0, 0),
    ([64, 65], [64, 1000], 4, 1, 128, 128, 0, 0),
    ([300, 1, 17], [300, 2500, 1040], 8, 2, 128, 32, 0, 0),
    ([257], [2257], 1, 1, 64, 512, 0, 0),
    ([200, 130], [3000, 130], 6, 2, 64, 16, 33, 5),
    ([50, 66], [1500, 80], 66, 2, 128, 16, 0, 0),
    ([20], [900], 128, 1, 64, 64, 0, 0),
    ([40], [9000], 60, 60, 64, 64, 0, 0),                       # long parts and a short one
    ([1024], [1324], 2, 1, 128, 16, 0, 0),
    ([500, 300], [3500, 301], 4, 2, 64, 32, 9, 330),
]


@pytest.mark.parametrize("new,lens,H,Hkv,d,page,window,sinks", CASES)
@pytest.mark.parametrize("shape", tr.SHAPES)
def test_tree_matches_definition(ralib, gpu, new, lens, H, Hkv, d, page, window, sinks, shape):
    c = Cache(lens, page, Hkv, d, sum(lens) + H)
    c.fill_all()
    q = randn_bf16((sum(new), H, d), 99 + H).cuda()
    trees = trees_of(new, shape)
    o_dtype = torch.float32 if shape == "bush" else torch.bfloat16
    o, lse, _ = attend(ralib, c, q, cu_of(new), trees, o_dtype, window, sinks)
    assert_trees(c, q, o, lse, trees, window, sinks)


@pytest.mark.parametrize("new,lens,H,Hkv,d,window", [
    ([8, 3], [900, 5000], 8, 2, 128, 0), ([70, 33], [900, 3000], 8, 2, 128, 0), ([32, 20], [2000, 20], 4, 4, 64, 100)])
def test_a_chain_is_the_causal_call(ralib, gpu, new, lens, H, Hkv, d, window):
    """A tree that is one token after another sees what ra_paged_attn_fwd's rows see: both within their
    tolerance of the definition, which is the same."""
    c = Cache(lens, 16, Hkv, d, 5)
    c.fill_all()
    q = randn_bf16((sum(new), H, d), 4).cuda()
    trees = trees_of(new, "chain")
    o, lse, ws = attend(ralib, c, q, cu_of(new), trees, torch.bfloat16, window)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    big = ralib.new_workspace(64 << 20)
    ralib.ra_paged_attn_fwd(q, c.k, c.v, c.table, c.seq_lens, cu_of(new), o2, lse2, max(new), max(lens), window, 0, workspace=big)
    for x, y in ((o, lse), (o2, lse2)):
        assert_trees(c, q, x, y, trees, window, 0)


@pytest.mark.parametrize("max_len", [1, 1 << 20])
@pytest.mark.parametrize("n", [2, 9, 40])
def test_any_guess_of_the_length(ralib, gpu, n, max_len):
    new, lens = [n, n], [6000, 77]
    c = Cache(lens, 32, 2, 128, 5)
    c.fill_all()
    q = randn_bf16((sum(new), 8, 128), 4).cuda()
    trees = trees_of(new, "forest")
    o, lse, _ = attend(ralib, c, q, cu_of(new), trees, torch.bfloat16, max_len=max_len)
    assert_trees(c, q, o, lse, trees, 0, 0)


@pytest.mark.parametrize("n", [3, 20])
@pytest.mark.parametrize("d", [64, 128])
def test_strides_padding_and_no_lse(ralib, gpu, n, d):
    """q as a part of a fused projection with padded rows of NaN around the sequences', which are left as
    they were; K and V of a page in one block; no LSE asked for."""
    new, lens, H, Hkv = [n, n, n], [400, n, 2000], 8, 2
    c = Cache(lens, 16, Hkv, d, 6, interleaved=True)
    c.fill_all()
    fused = torch.full((3 * n + 12, H + 2 * Hkv, d), NAN, dtype=torch.bfloat16, device="cuda")
    fused[3:3 + 3 * n] = randn_bf16((3 * n, H + 2 * Hkv, d), 8).cuda()
    q = fused[:, :H]
    trees = trees_of(new, "levels")
    for lse in (True, False):
        o, l, _ = attend(ralib, c, q, cu_of(new, 3), trees, torch.bfloat16, first=3, lse=lse)
        assert_trees(c, q, o, l, trees, 0, 0, first=3)
        assert bool(torch.isnan(o[:3]).all()) and bool(torch.isnan(o[3 + 3 * n:]).all())
        assert not lse or bool(torch.isnan(l[:, :3]).all()) and bool(torch.isnan(l[:, 3 + 3 * n:]).all())


@pytest.mark.parametrize("n", [8, 40])
def test_window_does_not_read_freed_pages(ralib, gpu, n):
    window, sinks, page, length = 300, 4, 32, 5000
    c = Cache([length], page, 2, 128, 12)
    c.fill_all()
    gone = torch.arange(1, (length - n - window) // page)
    c.table[0, gone] = -1
    q = randn_bf16((n, 8, 128), 3).cuda()
    trees = trees_of([n], "bush")
    o, lse, _ = attend(ralib, c, q, cu_of([n]), trees, torch.bfloat16, window, sinks)
    assert_trees(c, q, o, lse, trees, window, sinks)


@pytest.mark.parametrize("n", [7, 40])
def test_what_is_no_tree_is_reported(ralib, gpu, n):
    """Parents out of their range count as -1 and are reported; so are lengths and pages, and the next
    call is fine.  More new tokens than the sequence is long: the places that exist are seen."""
    new, lens, H, d = [n, n], [500, 800], 8, 128
    c = Cache(lens, 16, 2, d, 13, extra_cols=0)
    c.fill_all()
    q = randn_bf16((2 * n, H, d), 3).cuda()
    trees = trees_of(new, "levels")
    ws = attend(ralib, c, q, cu_of(new), trees, torch.bfloat16)[2]
    for bad in (-2, 4, n, 2 ** 31 - 1, -2 ** 31):
        raw = flat(trees)
        raw[n + 4] = bad
        o, lse, _ = attend(ralib, c, q, cu_of(new), trees, torch.bfloat16, ws=ws, check=False, parents=raw)
        with pytest.raises(ralib.RAError, match="tree|lengths|page"):
            ralib.ra_check_status(ws)
        as_root = [trees[0], trees[1][:4] + [-1] + trees[1][5:]]
        assert_trees(c, q, o, lse, as_root, 0, 0)
    good = c.table.clone()
    c.table[1, 3] = c.n_pages
    attend(ralib, c, q, cu_of(new), trees, torch.bfloat16, ws=ws, check=False)
    with pytest.raises(ralib.RAError):
        ralib.ra_check_status(ws)
    c.table.copy_(good)
    for length in (0, n - 2, -3, 10 ** 6):
        c.seq_lens[0] = length
        o, lse, _ = attend(ralib, c, q, cu_of(new), trees, torch.bfloat16, ws=ws, check=False)
        with pytest.raises(ralib.RAError):
            ralib.ra_check_status(ws)
        if length <= 0:
            assert bool((o[:n] == 0).all()) and bool(torch.isneginf(lse[:, :n]).all())
    c.seq_lens.copy_(torch.tensor(lens))
    o, lse, _ = attend(ralib, c, q, cu_of(new), trees, torch.bfloat16, ws=ws)
    assert_trees(c, q, o, lse, trees, 0, 0)


@pytest.mark.parametrize("n", [6, 25])
def test_scores_far_from_zero(ralib, gpu, n):
    """Scores near 0, far below and far above, among the context and among the new tokens."""
    lens, H, d = [9000], 8, 128
    c = Cache(lens, 64, 1, d, 17)
    q = randn_bf16((n, H, d), 3).cuda()
    q[..., 0] = 16.0
    c.ks[0][..., 0] = -30.0
    c.ks[0][1000:1004, :, 0] = 25.0
    c.ks[0][8999 - n // 2, :, 0] = 27.0
    c.fill_all()
    trees = trees_of([n], "levels")
    o, lse, _ = attend(ralib, c, q, cu_of([n]), trees, torch.float32)
    oe, le, p, vd = expect(c, q, trees[0], 0, 0, 0, 0)
    # a score's 32-bit sum here is as large as 16 * 30 and off by up to 2e-4 more
    ref.assert_within(o[None], oe, 2 * ref.forward_tolerance(p, vd, oe, False), "O")
    ref.assert_within(lse[None], le, 1e-5 * le.abs() + 4 * ref.EPS, "LSE")


@pytest.mark.parametrize("new_max,longest", [(8, 3000), (8, 900), (90, 3000)])
def test_many_sequences(ralib, gpu, new_max, longest):
    """More units than multiprocessors, sequences without new tokens among them; the same bits again."""
    r = random.Random(new_max)
    new = [r.randint(0, new_max) for _ in range(70)]
    lens = [x + r.randint(0, longest) for x in new]
    c = Cache(lens, 64, 8, 128, 71)
    c.fill_all()
    q = randn_bf16((sum(new), 32, 128), 5).cuda()
    trees = trees_of(new, "levels")
    o, lse, ws = attend(ralib, c, q, cu_of(new), trees, torch.bfloat16)
    assert_trees(c, q, o, lse, trees, 0, 0)
    again = attend(ralib, c, q, cu_of(new), trees, torch.bfloat16, ws=ws)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("new,longest,H,Hkv,d", [
    ([8] * 100, 900, 16, 8, 64), ([8] * 70, 3000, 16, 8, 64), ([8, 3], 9000, 8, 2, 128), ([16, 3], 20000, 8, 4, 128),
    ([40], 20000, 8, 2, 128), ([40, 2, 300], 700, 8, 2, 64), ([60, 2, 60], 100, 8, 2, 64)])
def test_workspace_is_not_left(ralib, gpu, new, longest, H, Hkv, d):
    """Nothing is written past the bytes a call asks for, and any words in them serve (its header apart)."""
    r = random.Random(longest)
    lens = [longest] + [max(x, r.randint(1, longest)) for x in new[1:]]
    c = Cache(lens, 16, Hkv, d, 91)
    c.fill_all()
    q = randn_bf16((sum(new), H, d), 4).cuda()
    need = ralib.ra_paged_tree_attn_workspace_bytes(sum(new), len(new), H, Hkv, d, max(new), longest)
    room = torch.zeros(need + (1 << 20), dtype=torch.uint8, device="cuda")
    room[256:] = 0xA5
    trees = trees_of(new, "forest")
    o, lse, _ = attend(ralib, c, q, cu_of(new), trees, torch.bfloat16, ws=room[:need])
    assert bool((room[need:] == 0xA5).all())
    assert_trees(c, q, o, lse, trees, 0, 0)


@pytest.mark.parametrize("n,length,window", [(3, 3000, 0), (40, 3000, 0), (40, 3000, 20)])
def test_pool_past_32_bits(ralib, gpu, n, length, window):
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
    c.fill_all()
    q = randn_bf16((n, H, d), 3).cuda()
    trees = trees_of([n], "levels")
    o, lse, _ = attend(ralib, c, q, cu_of([n]), trees, torch.bfloat16, window, 4 if window else 0)
    assert_trees(c, q, o, lse, trees, window, 4 if window else 0)


def test_binding_refuses(ralib, gpu):
    c = Cache([100], 16, 2, 64, 37)
    q = randn_bf16((3, 4, 64), 1).cuda()
    o, cu, ws = torch.empty_like(q), cu_of([3]), ralib.new_workspace(256)
    par = flat([[-1, 0, 0]])

    def call(**kw):
        a = dict(q=q, k=c.k, v=c.v, par=par, cu=cu, o=o, ws=ws, new=3)
        a.update(kw)
        ralib.ra_paged_tree_attn_fwd(a["q"], a["k"], a["v"], c.table, c.seq_lens, a["cu"], a["par"], a["o"], None, a["new"], 100,
                                     workspace=a["ws"])

    for kw in (dict(q=q.half()), dict(par=par.long()), dict(o=o.half()), dict(par=None)):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(par=par[:2]), dict(par=par.cpu()), dict(cu=cu[:1]), dict(ws=None), dict(o=o[:, :2])):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ralib.RAError):
        call(new=1025)


@pytest.mark.parametrize("H,Hkv,d", [(9, 3, 128), (10, 5, 64), (7, 7, 128), (22, 11, 64), (24, 12, 128), (40, 1, 64)])
def test_head_counts(ralib, gpu, H, Hkv, d):
    """Key/value heads whose lists do not divide the GPU evenly, or are several heads long."""
    new, lens = [33, 40, 2, 60], [700, 4000, 300, 61]
    c = Cache(lens, 32, Hkv, d, 43)
    c.fill_all()
    q = randn_bf16((sum(new), H, d), 44).cuda()
    trees = trees_of(new, "levels")
    o, lse, _ = attend(ralib, c, q, cu_of(new), trees, torch.bfloat16)
    assert_trees(c, q, o, lse, trees, 0, 0)


@pytest.mark.parametrize("n,longest,new_max", [(40, 900, 40), (500, 200, 40), (1200, 60, 3), (33, 9000, 8)])
def test_many_sequences_in_runs(ralib, gpu, n, longest, new_max):
    """More sequences than a warp or a block has threads, most of them without new tokens."""
    r = random.Random(n)
    new = [r.choice([0, 0, r.randint(1, new_max)]) for _ in range(n)]
    new[n // 2] = new_max
    lens = [x + r.randint(0, longest) for x in new]
    c = Cache(lens, 16, 4, 64, 73)
    c.fill_all()
    q = randn_bf16((sum(new), 16, 64), 5).cuda()
    trees = trees_of(new, "forest")
    for max_len in (max(lens), 1 << 22):
        o, lse, _ = attend(ralib, c, q, cu_of(new), trees, torch.bfloat16, max_len=max_len)
        assert_trees(c, q, o, lse, trees, 0, 0)


def test_sequences_that_see_nothing_among_others(ralib, gpu):
    """A sequence shorter than its new tokens in the middle of a run: its rows before place 0 are
    empty, the others are the definition's."""
    new, lens, H, d = [40, 50, 33], [900, 50, 1200], 8, 64
    c = Cache(lens, 16, 2, d, 47)
    c.fill_all()
    q = randn_bf16((sum(new), H, d), 3).cuda()
    trees = trees_of(new, "star")
    c.seq_lens[1] = 0
    o, lse, _ = attend(ralib, c, q, cu_of(new), trees, torch.bfloat16, check=False)
    assert bool((o[40:90] == 0).all()) and bool(torch.isneginf(lse[:, 40:90]).all())
    good = Cache.__new__(Cache)
    for s, at in ((0, 0), (2, 90)):
        good.lens, good.ks, good.vs = [lens[s]], [c.ks[s]], [c.vs[s]]
        rows = slice(at, at + new[s])
        assert_trees(good, q[rows], o[rows], lse[:, rows], [trees[s]], 0, 0)


@pytest.mark.parametrize("n", [8, 40])
def test_two_graphs_share_a_workspace(ralib, gpu, n):
    """Two captured calls of different sizes, replayed in turns on one workspace, and an eager one between."""
    shapes = [([n, n], [5000, 700], 8, 2, 128), ([n], [20000], 16, 4, 64)]
    ws = ralib.new_workspace(64 << 20)
    work = []
    for new, lens, H, Hkv, d in shapes:
        c = Cache(lens, 32, Hkv, d, 51)
        c.fill_all()
        q = randn_bf16((sum(new), H, d), 7).cuda()
        trees = trees_of(new, "levels")
        o, lse = torch.empty_like(q), torch.empty((H, sum(new)), device="cuda")
        args = (q, c.k, c.v, c.table, c.seq_lens, cu_of(new), flat(trees), o, lse, max(new), max(lens))
        ralib.ra_paged_tree_attn_fwd(*args, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            ralib.ra_paged_tree_attn_fwd(*args, workspace=ws)
        work.append((c, q, o, lse, trees, graph, args))
    for i in range(6):
        c, q, o, lse, trees, graph, args = work[i % 2]
        o.fill_(NAN)
        graph.replay()
        if i > 2:
            ralib.ra_paged_tree_attn_fwd(*work[1 - i % 2][6], workspace=ws)
        ralib.ra_check_status(ws)
        assert_trees(c, q, o, lse, trees, 0, 0)


@pytest.mark.parametrize("n", [8, 40])
def test_two_streams_two_workspaces(ralib, gpu, n):
    new, lens = [n] * 3, [20000, 300, 7000]
    c = Cache(lens, 64, 2, 128, 83)
    c.fill_all()
    q = randn_bf16((3 * n, 8, 128), 4).cuda()
    trees = trees_of(new, "bush")
    want, want_lse, _ = attend(ralib, c, q, cu_of(new), trees, torch.bfloat16)
    cu, parents = cu_of(new), flat(trees)
    outs = [(torch.cuda.Stream(), torch.empty_like(want), torch.empty_like(want_lse), ralib.new_workspace(48 << 20)) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o, lse, ws in outs:
            ralib.ra_paged_tree_attn_fwd(q, c.k, c.v, c.table, c.seq_lens, cu, parents, o, lse, n, max(lens), workspace=ws, stream=s)
    torch.cuda.synchronize()
    for _, o, lse, ws in outs:
        ralib.ra_check_status(ws)
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
