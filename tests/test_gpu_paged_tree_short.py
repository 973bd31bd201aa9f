"""Calls on trees whose sequences break their bounds, against the definition: sequences shorter than their
new rows, whose rows see what of their ancestors lies in the cache, and parents that are none, which
count as roots.  And how often the few-row form of tree attention rounds its weights."""
import pytest
import torch

import tree_reference as tr
import window_reference as ref
from synthetic_inputs import randn_bf16
from test_gpu_paged import Cache, cu_of
from test_gpu_paged_keep import expect as kept, ints, keep, make
from test_gpu_paged_tree import attend, expect, trees_of
from test_gpu_roundings import rounded, two_part_tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,H,Hkv,d", [(7, 8, 2, 128), (25, 4, 4, 64), (8, 8, 2, 64), (40, 8, 2, 128), (300, 4, 1, 64), (130, 6, 2, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (5, 4)])
@pytest.mark.parametrize("shape", ["levels", "chain", "forest"])
def test_sequences_shorter_than_their_new_rows(ralib, gpu, n, H, Hkv, d, window, sinks, shape):
    """Places before 0 are not there: a row at one may still have ancestors or itself in the cache, or nothing."""
    other = 50
    for length in sorted({n - 1, n - 2, n // 2, 1}):
        c = Cache([max(length, 1), 400], 16, Hkv, d, 13)
        c.fill_all()
        new = [n, other]
        trees = trees_of(new, shape)
        q = randn_bf16((sum(new), H, d), 3).cuda()
        o, lse, ws = attend(ralib, c, q, cu_of(new), trees, torch.float32, window, sinks, check=False)
        with pytest.raises(ralib.RAError):
            ralib.ra_check_status(ws)
        # the definition over a cache that begins n - length places before it: those places are seen by nobody
        t0 = 0
        for s, tree in enumerate(trees):
            m, before = len(tree), c.lens[s] - len(tree)
            ok = torch.zeros((m, c.lens[s]), dtype=torch.bool)
            for i, places in enumerate(tr.sees(tree, before, window, sinks)):
                ok[i, sorted(places)] = True
            kd, vd = (ref.expand_kv(x[s].double()[None], H) for x in (c.ks, c.vs))
            oe, le, p = ref.forward(q[t0:t0 + m].double()[None], kd, vd, ok.cuda(), d ** -0.5)
            ref.assert_within(o[t0:t0 + m][None], oe, ref.forward_tolerance(p, vd, oe, False), "length %d sequence %d O" % (length, s))
            empty = torch.isneginf(le[0])
            got = lse[:, t0:t0 + m]
            assert torch.equal(torch.isneginf(got), empty), (length, s)
            ref.assert_within(got[~empty], le[0][~empty], torch.full_like(le[0][~empty], ref.EPS), "length %d sequence %d LSE" % (length, s))
            t0 += m


@pytest.mark.parametrize("bad", [5, 19, -2, 2 ** 31 - 1, -2 ** 31])
def test_a_bad_parent_on_the_path_is_a_root(ralib, gpu, bad):
    """ra_paged_keep_path over parents that are none: the node counts as a root, its path begins there."""
    trees, lens = [tr.random_tree(20, "levels", 1), tr.random_tree(9, "bush", 2)], [100, 60]
    at = [i for i in tr.path(trees[0], 19) if i >= 3][0]          # a node on the way to the last
    bad = at if bad == 5 else bad                                # (its own number; one behind it; ..)
    c = make(lens, 16, 2, 64, 2, 5)
    raw = ints(trees[0] + trees[1])
    raw[at] = bad
    as_root = [trees[0][:at] + [-1] + trees[0][at + 1:], trees[1]]
    want, lens_e, rows_e = kept(c, as_root, [19, 8])
    new_lens, rows, ws = keep(ralib, c, trees, [19, 8], check=False, raw=raw)
    with pytest.raises(ralib.RAError):
        ralib.ra_check_status(ws)
    assert new_lens.tolist() == lens_e and rows.tolist() == rows_e
    for s, n in enumerate(lens_e):
        p, place = c.places(s, 0, n)
        for x, y in zip(c.pools, want):
            assert torch.equal(x[:, p, place], y[:, p, place])


@pytest.mark.parametrize("new,lens,H,Hkv,d,window,sinks", [
    ([4, 1, 2], [4, 1, 40], 8, 2, 128, 0, 0),                       # 16 rows: a cluster to a pair
    ([8, 3, 5], [9, 3, 300], 8, 2, 128, 0, 0),                      # 32 rows in blocks of 16
    ([8, 2], [3000, 2], 8, 2, 64, 0, 0),
    ([2] * 100, [2 + i % 5 for i in range(100)], 8, 2, 64, 0, 0),   # a block to a pair
    ([32, 7], [32, 9], 4, 4, 64, 2, 1),
])
def test_few_rows_round_their_weights_twice(ralib, gpu, new, lens, H, Hkv, d, window, sinks):
    """The bound of P in two bf16 parts (test_gpu_roundings.py), which P in one part would break."""
    c = Cache(lens, 16, Hkv, d, sum(lens) + d)
    c.fill_all()
    q = randn_bf16((sum(new), H, d), 41).cuda()
    trees = trees_of(new, "bush")
    o, _, _ = attend(ralib, c, q, cu_of(new), trees, torch.float32, window, sinks)
    t0, beyond = 0, False
    for s, n in enumerate(new):
        o_ref, _, p, vd = expect(c, q, trees[s], s, t0, window, sinks)
        tol = two_part_tolerance(p, vd, o_ref)
        ref.assert_within(o[t0:t0 + n][None], o_ref, tol, "sequence %d" % s)
        beyond = beyond or bool(((torch.einsum("bhlt,bthd->blhd", rounded(p), vd) - o_ref).abs() > tol).any())
        t0 += n
    assert beyond, "the bound would pass P in one bf16 value"
