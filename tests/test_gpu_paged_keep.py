"""Keeping the accepted path of a tree in a paged cache, and a round of drafting as a server runs it."""
import random

import pytest
import torch

import tree_reference as tr
from synthetic_inputs import randn_bf16
from test_gpu_readme import snippet
from test_gpu_paged import NAN, Cache, cu_of
from test_gpu_paged_rotary import frequencies, rotated
from test_gpu_paged_tree import assert_trees

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(lens, page, Hkv, d, layers, seed, side_by_side=False):
    c = Cache(lens, page, Hkv, d, seed)
    shape = (layers, c.n_pages, page, Hkv, d)
    c.pools = []
    for i in range(2):
        x = randn_bf16(shape, seed + i).cuda()
        if side_by_side:       # the layers' pages beside one another
            y = torch.empty((c.n_pages, layers, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
            y.copy_(x.transpose(0, 1))
            x = y.transpose(0, 1)
        c.pools.append(x)
    return c


def expect(c, trees, last, first=0):
    """The pools, lengths and path that the definition gives."""
    pools = [x.clone() for x in c.pools]
    lens, rows, t0 = [], [-1] * sum(len(t) for t in trees), 0
    for s, (tree, leaf) in enumerate(zip(trees, last)):
        path, before = tr.path(tree, leaf), c.lens[s] - len(tree)
        if path:
            src = c.table[s].long()[(before + torch.tensor(path)).cuda() // c.page], (before + torch.tensor(path)).cuda() % c.page
            dst = c.places(s, before, before + len(path))
            for x, y in zip(pools, c.pools):
                x[:, dst[0], dst[1]] = y[:, src[0], src[1]]
        lens.append(before + len(path))
        for j, a in enumerate(path):
            rows[t0 + j] = first + t0 + a
        t0 += len(tree)
    return pools, lens, rows


def keep(ra, c, trees, last, first=0, tail=0, path=True, check=True, raw=None, pools=None):
    n = sum(len(t) for t in trees)
    parents = ints([3] * first + [x for t in trees for x in t] + [-8] * tail) if raw is None else raw
    new_lens = torch.full((len(trees),), -77, dtype=torch.int32, device="cuda")
    rows = torch.full((first + n + tail,), -77, dtype=torch.int32, device="cuda") if path else None
    ws = ra.new_workspace(256)
    k, v = c.pools if pools is None else pools
    ra.ra_paged_keep_path(k, v, c.table, c.seq_lens, cu_of([len(t) for t in trees], first), parents, ints(last), new_lens, rows,
                          workspace=ws)
    if check:
        ra.ra_check_status(ws)
    return new_lens, rows, ws


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("shape", tr.SHAPES)
@pytest.mark.parametrize("new,extra,Hkv,d,page,layers", [
    ([1], [0], 1, 64, 16, 1),
    ([26, 0, 60, 8], [974, 5, 0, 33], 2, 128, 16, 3),
    ([40] * 9, [7 * i for i in range(9)], 8, 64, 32, 5),
    ([1024, 300], [10, 100], 1, 64, 64, 2),
    ([20] * 300, [i for i in range(300)], 1, 128, 16, 2),
])
@pytest.mark.parametrize("side_by_side", [False, True])
def test_keep_path(ralib, gpu, new, extra, Hkv, d, page, layers, shape, side_by_side):
    lens = [a + b for a, b in zip(new, extra)]
    c = make(lens, page, Hkv, d, layers, 7, side_by_side)
    trees = [tr.random_tree(n, shape, 11 + i) for i, n in enumerate(new)]
    r = random.Random(len(new))
    last = [r.choice([-1, n - 1, r.randint(-1, n - 1)]) if n else -1 for n in new]
    last[0] = new[0] - 1
    want, lens_e, rows_e = expect(c, trees, last, first=2)
    new_lens, rows, _ = keep(ralib, c, trees, last, first=2, tail=3)
    assert new_lens.tolist() == lens_e
    assert rows.tolist() == [-77] * 2 + rows_e + [-77] * 3
    for x, y in zip(c.pools, want):
        # places behind the path hold anything: what was there, or a node that moved down
        for s, n in enumerate(lens_e):
            p, at = c.places(s, n, lens[s])
            x[:, p, at] = y[:, p, at] = 0
        assert same(x, y)


def test_one_pool_and_no_path(ralib, gpu):
    """A pool without layers; path not asked for; places overlap along the whole chain."""
    c = make([300], 16, 2, 64, 1, 9)
    tree = [-1, -1] + list(range(1, 79))           # node 1, then a chain: every node moves down by one
    want, lens, _ = expect(c, [tree], [79])
    new_lens, _, _ = keep(ralib, c, [tree], [79], path=False, pools=[x[0] for x in c.pools])
    assert new_lens.tolist() == lens == [299]
    p, at = c.places(0, 0, 299)
    for x, y in zip(c.pools, want):
        assert torch.equal(x[:, p, at], y[:, p, at])


def test_what_is_no_path_is_reported(ralib, gpu):
    trees, lens = [tr.random_tree(20, "levels", 1), tr.random_tree(9, "bush", 2)], [100, 60]
    c = make(lens, 16, 2, 64, 2, 5)
    before = [x.clone() for x in c.pools]
    for bad in (9, -2, 2 ** 31 - 1, -2 ** 31):
        c.pools = [x.clone() for x in before]
        want, lens_e, rows_e = expect(c, trees, [19, -1])
        new_lens, rows, ws = keep(ralib, c, trees, [19, bad], check=False)
        with pytest.raises(ralib.RAError, match="tree"):
            ralib.ra_check_status(ws)
        assert new_lens.tolist() == lens_e and rows.tolist() == rows_e
        p, at = c.places(0, 0, lens_e[0])
        p2, at2 = c.places(1, 0, lens[1])
        for x, y in zip(c.pools, want):
            assert torch.equal(x[:, p, at], y[:, p, at]) and torch.equal(x[:, p2, at2], y[:, p2, at2])
    # parents that are none, a page outside the pool, more nodes than the length, a length past the table
    raw = ints(trees[0] + trees[1])
    raw[5] = 5
    _, _, ws = keep(ralib, c, trees, [19, 8], check=False, raw=raw)
    with pytest.raises(ralib.RAError):
        ralib.ra_check_status(ws)
    good = c.table.clone()
    c.table[0, 99 // 16] = c.n_pages
    _, _, ws = keep(ralib, c, trees, [19, 8], check=False)
    with pytest.raises(ralib.RAError):
        ralib.ra_check_status(ws)
    c.table.copy_(good)
    for length, then in ((12, 0), (-5, 0), (10 ** 6, None)):
        c.seq_lens[0] = length
        c.pools = [x.clone() for x in before]
        new_lens, _, ws = keep(ralib, c, trees, [19, -1], check=False)
        with pytest.raises(ralib.RAError):
            ralib.ra_check_status(ws)
        assert then is None or new_lens.tolist()[0] == then
        p, at = c.places(0, 0, lens[0])
        for x, y in zip(c.pools, before):
            assert torch.equal(x[:, p, at], y[:, p, at])


def test_pool_past_32_bits(ralib, gpu):
    page, Hkv, d, layers = 256, 8, 128, 3
    c = Cache([1000], page, Hkv, d, 5)
    n_pages = (1 << 31) // (page * Hkv * d) + 20
    c.pools = [torch.empty((layers, n_pages, page, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    c.n_pages = n_pages
    c.table[0, :4] = ints([n_pages - 1, n_pages - 9, n_pages - 4, n_pages - 2])
    tree = tr.random_tree(60, "levels", 4)
    path = tr.path(tree, 59)
    p, at = c.places(0, 940, 1000)
    data = [randn_bf16((layers, 60, Hkv, d), 3 + i).cuda() for i in range(2)]
    for x, y in zip(c.pools, data):
        x[:, p, at] = y
    new_lens, _, _ = keep(ralib, c, [tree], [59])
    assert new_lens.tolist() == [940 + len(path)]
    for x, y in zip(c.pools, data):
        assert torch.equal(x[:, p[:len(path)], at[:len(path)]], y[:, torch.tensor(path).cuda()])


def test_binding_refuses(ralib, gpu):
    c = make([50], 16, 1, 64, 2, 3)
    tree = [-1, 0, 0]
    par, last, lens, cu = ints(tree), ints([2]), torch.empty_like(c.seq_lens), cu_of([3])
    ws = ralib.new_workspace(256)

    def call(**kw):
        a = dict(k=c.pools[0], v=c.pools[1], par=par, last=last, lens=lens, path=None, ws=ws)
        a.update(kw)
        ralib.ra_paged_keep_path(a["k"], a["v"], c.table, c.seq_lens, cu, a["par"], a["last"], a["lens"], a["path"], workspace=a["ws"])

    for kw in (dict(k=c.pools[0].float()), dict(par=par.long()), dict(last=last.long()), dict(lens=None)):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(v=c.pools[1][0]), dict(last=ints([1, 1])), dict(lens=ints([])), dict(path=ints([0, 0])), dict(par=par[None]),
               dict(last=last.cpu()), dict(ws=None), dict(k=c.pools[0][:0], v=c.pools[1][:0])):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ralib.RAError):
        call(lens=c.seq_lens)
    with pytest.raises(ralib.RAError):        # the layers' pages would be one another's
        call(k=c.pools[0][:1].expand(2, -1, -1, -1, -1), v=c.pools[1][:1].expand(2, -1, -1, -1, -1))


@pytest.mark.parametrize("H,Hkv,d,n_draft", [(8, 2, 128, 7), (4, 4, 64, 40)])
def test_rounds_of_drafting_replayed(ralib, gpu, H, Hkv, d, n_draft):
    """Append with rotation, attend, keep -- captured once and replayed over several rounds with other trees,
    accepted nodes and tokens.  Each round's outputs are the definition's over the tokens kept so far, and a
    round run without the graph on the same state gives the same bits."""
    page, n, rounds, pairs = 16, 3, 5, d == 64
    start = [33, 5, 200]
    room = [x + rounds * (n_draft + 1) + n_draft for x in start]
    c = Cache(room, page, Hkv, d, 23)
    freq = frequencies(d // 2)
    raw_k = [randn_bf16((x, Hkv, d), 60 + s).cuda() for s, x in enumerate(start)]
    c.vs = [randn_bf16((x, Hkv, d), 70 + s).cuda() for s, x in enumerate(start)]
    ws = ralib.new_workspace(64 << 20)
    # the prompts
    c.seq_lens.copy_(ints(start))
    q0 = randn_bf16((sum(start), H, d), 5).cuda()
    ralib.ra_paged_append_rotary(q0, torch.cat(raw_k), torch.cat(c.vs), q0, c.k, c.v, c.table, c.seq_lens, cu_of(start), freq,
                                 pairs=pairs, workspace=ws)
    c.lens = list(start)
    c.ks = [c.k[c.places(s, 0, x)] for s, x in enumerate(start)]
    for s, x in enumerate(start):
        e, t = rotated(raw_k[s], torch.arange(x, device="cuda"), freq, pairs)
        assert bool(((c.ks[s].double() - e).abs() <= t).all())
    T = n * n_draft
    qkv = torch.empty((T, H + 2 * Hkv, d), dtype=torch.bfloat16, device="cuda")
    q, kn, vn = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    qr = torch.empty((T, H, d), dtype=torch.bfloat16, device="cuda")
    o, lse = torch.empty_like(qr), torch.empty((H, T), device="cuda")
    parents, last, new_lens, path = ints([-1] * T), ints([-1] * n), ints([0] * n), ints([0] * T)
    cu, max_len = cu_of([n_draft] * n), max(room)

    def step():
        ralib.ra_paged_append_rotary(q, kn, vn, qr, c.k, c.v, c.table, c.seq_lens, cu, freq, parents=parents, pairs=pairs,
                                     workspace=ws)
        ralib.ra_paged_tree_attn_fwd(qr, c.k, c.v, c.table, c.seq_lens, cu, parents, o, lse, n_draft, max_len, workspace=ws)
        ralib.ra_paged_keep_path(c.k, c.v, c.table, c.seq_lens, cu, parents, last, new_lens, path, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    r = random.Random(1)
    for i in range(rounds):
        trees = [tr.random_tree(n_draft, tr.SHAPES[(i + s) % 5], i + s) for s in range(n)]
        leaves = [r.randint(-1, n_draft - 1) for _ in range(n)]
        parents.copy_(ints([x for t in trees for x in t]))
        last.copy_(ints(leaves))
        qkv.copy_(randn_bf16(tuple(qkv.shape), 100 + i).cuda())
        before = list(c.lens)
        c.seq_lens.copy_(ints([x + n_draft for x in before]))
        state = c.k.clone(), c.v.clone()
        graph.replay()
        once = o.clone(), lse.clone(), c.k.clone(), c.v.clone(), new_lens.clone(), path.clone(), qr.clone()
        c.k.copy_(state[0])
        c.v.copy_(state[1])
        ralib.ra_paged_append_rotary(q, kn, vn, qr, c.k, c.v, c.table, c.seq_lens, cu, freq, parents=parents, pairs=pairs,
                                     workspace=ws)
        drafts = [c.k[c.places(s, before[s], before[s] + n_draft)] for s in range(n)]
        step()
        for x, y in zip((o, lse, c.k, c.v, new_lens, path, qr), once):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        ralib.ra_check_status(ws)
        # the definition: the tokens kept so far, and the drafts as they were rotated
        pos = [b + len(tr.path(t, j)) - 1 for b, t in zip(before, trees) for j in range(n_draft)]
        pos = torch.tensor(pos, device="cuda")
        qe, qt = rotated(q, pos, freq, pairs)
        assert bool(((qr.double() - qe).abs() <= qt).all())
        for s in range(n):
            rows = slice(s * n_draft, (s + 1) * n_draft)
            e, t = rotated(kn[rows], pos[rows], freq, pairs)
            assert bool(((drafts[s].double() - e).abs() <= t).all())
        full = Cache.__new__(Cache)
        full.lens = [b + n_draft for b in before]
        full.ks = [torch.cat([c.ks[s], drafts[s]]) for s in range(n)]
        full.vs = [torch.cat([c.vs[s], vn[s * n_draft:(s + 1) * n_draft]]) for s in range(n)]
        assert_trees(full, qr, o, lse, trees, 0, 0)
        for s in range(n):
            p = tr.path(trees[s], leaves[s])
            assert int(new_lens[s]) == before[s] + len(p)
            assert path[s * n_draft:(s + 1) * n_draft].tolist() == [s * n_draft + a for a in p] + [-1] * (n_draft - len(p))
            c.lens[s] = before[s] + len(p)
            now = c.places(s, before[s], c.lens[s])
            at = torch.tensor(p, dtype=torch.long, device="cuda")
            e, t = rotated(kn[s * n_draft:(s + 1) * n_draft][at], torch.arange(before[s], c.lens[s], device="cuda"), freq, pairs)
            assert bool(((c.k[now].double() - e).abs() <= t).all())
            assert torch.equal(c.v[now], vn[s * n_draft:(s + 1) * n_draft][at])
            old = c.places(s, 0, before[s])
            assert torch.equal(c.k[old], c.ks[s]) and torch.equal(c.v[old], c.vs[s])
            c.ks[s] = c.k[c.places(s, 0, c.lens[s])]
            c.vs[s] = c.v[c.places(s, 0, c.lens[s])]


def test_a_server_follows_the_readme(ralib, gpu):
    """The README's snippet, as it stands there."""
    n, H, H_kv, d, page, new = 3, 8, 4, 128, 16, [12, 1, 30]
    lens = [1000, 40, 300]
    c = Cache(lens, page, H_kv, d, 11)
    for s, (x, length) in enumerate(zip(new, lens)):
        c.fill(s, 0, length - x)
    trees = [tr.random_tree(x, tr.SHAPES[s], s) for s, x in enumerate(new)]
    T = sum(new)
    names = dict(ra=ralib, T=T, n=n, H=H, H_kv=H_kv, d=d, max_new=max(new), max_len=max(lens), k_pages=c.k, v_pages=c.v,
                 block_table=c.table, seq_lens=c.seq_lens, cu=cu_of(new), parents=ints([x for t in trees for x in t]),
                 q=randn_bf16((T, H, d), 5).cuda(), k_new=randn_bf16((T, H_kv, d), 6).cuda(),
                 v_new=randn_bf16((T, H_kv, d), 7).cuda(), inv_freq=frequencies(d // 2), last=ints([x - 1 for x in new]),
                 o=torch.empty((T, H, d), dtype=torch.bfloat16, device="cuda"), lse=torch.empty((H, T), device="cuda"),
                 q_rot=torch.empty((T, H, d), dtype=torch.bfloat16, device="cuda"), new_lens=ints([0] * n), path=ints([0] * T))
    lines = snippet("ra_paged_keep_path").split("# last: ")
    exec(lines[0], names)
    ks, vs = ([x[c.places(s, 0, m)] for s, m in enumerate(lens)] for x in (c.k, c.v))
    full = Cache.__new__(Cache)
    full.lens, full.ks, full.vs = lens, ks, vs
    assert_trees(full, names["q_rot"], names["o"], names["lse"], trees, 0, 0)
    exec("# " + lines[1], names)
    ralib.ra_check_status(names["ws"])
    for s, (x, m) in enumerate(zip(new, lens)):
        at = [m - x + a for a in tr.path(trees[s], x - 1)]
        assert int(names["new_lens"][s]) == m - x + len(at)
        now = c.places(s, m - x, m - x + len(at))
        assert torch.equal(c.k[now], ks[s][at]) and torch.equal(c.v[now], vs[s][at])
