"""Trees over very long contexts: units that take seconds, and long sums.  (A page serves many times in a
sequence's table, so the caches are small.)"""
import pytest
import torch

import tree_reference as tr
import window_reference as ref
from synthetic_inputs import randn_bf16
from test_gpu_paged import NAN, Cache, cu_of
from test_gpu_paged_tree import CASES, assert_trees, attend, trees_of

pytestmark = pytest.mark.gpu


def test_units_that_take_seconds(ralib, gpu):
    """320 nodes of 128 query heads over 2^28 keys: 160 units, about 3.4 s each, a little more than one to a
    multiprocessor.  Keys of zero: each weight is 1, and a row's sum a whole number of at most 2^28, off by less
    than 2^-20 of it in 32 bits.  Values of zero in the cache and +-2^j in the new rows: O is those times the
    row's nodes over all that it sees, whose rounding to bf16 is the larger part of its error."""
    H, d, n, page, length = 128, 64, 320, 65536, 1 << 28
    k = torch.zeros((2, page, 1, d), dtype=torch.bfloat16, device="cuda")
    row = torch.tensor([(-1.0) ** (i % 3) * 2.0 ** (i % 5 + 20) for i in range(d)], device="cuda").bfloat16()
    v = torch.zeros_like(k)
    v[1, page - n:] = row
    table = torch.zeros((1, length // page), dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    tree = tr.random_tree(n, "levels", 3)
    q = randn_bf16((n, H, d), 5).cuda()
    o = torch.full((n, H, d), NAN, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, n), NAN, device="cuda")
    ws = ralib.new_workspace(ralib.ra_paged_tree_attn_workspace_bytes(n, 1, H, 1, d, n, length))
    ralib.ra_paged_tree_attn_fwd(q, k, v, table, torch.tensor([length], dtype=torch.int32, device="cuda"), cu_of([n]),
                                 torch.tensor(tree, dtype=torch.int32, device="cuda"), o, lse, n, length, workspace=ws)
    ralib.ra_check_status(ws)
    nodes = torch.tensor([len(tr.path(tree, i)) for i in range(n)], dtype=torch.float64, device="cuda")
    seen = length - n + nodes
    want = (nodes / seen)[:, None, None] * row.double()
    assert bool(((o.double() - want).abs() <= (2.0 ** -9 + 2.0 ** -18) * want.abs()).all())
    # (the logarithm of about 2^28 in 32 bits: a few units of 2^-19)
    assert (lse.double() - seen.log()).abs().max().item() <= 1e-5


@pytest.mark.parametrize("n_seqs,n,H,d,lg", [
    (1, 320, 128, 64, 22), (1, 320, 128, 128, 22),      # two Q tiles, a unit and a bit to a multiprocessor
    (160, 20, 5, 128, 22),                              # one Q tile
    (2, 20, 5, 64, 24), (2, 200, 5, 128, 23)])          # cut units, each piece long
@pytest.mark.parametrize("window", [0, (1 << 21) + 77])
def test_long_sums(ralib, gpu, n_seqs, n, H, d, lg, window):
    """Values about 1, so that sums grow all along: a product cuts off less than 2^-21 of the sum it adds to, and
    1024 key tiles of eight products are added at a time, to half of their sum on average: 2^-9 of it in all.  The rounding of
    the weights to bf16 comes on top (the sum they are divided by has it too).  The keys' scale differs
    between the halves of the context, so that the references of the parts do."""
    page, length = 65536, 1 << lg
    pages = length // page
    k = randn_bf16((3, page, 1, d), 7).cuda()
    k[1] *= 1.5
    v = (1 + 0.25 * randn_bf16((3, page, 1, d), 8).float()).bfloat16().cuda()
    table = torch.zeros((n_seqs, pages), dtype=torch.int32, device="cuda")
    table[:, pages // 2:] = 1
    table[:, -1] = 2
    trees = [tr.random_tree(n, "levels", s) for s in range(n_seqs)]
    q = randn_bf16((n_seqs * n, H, d), 5).cuda()
    o = torch.full((n_seqs * n, H, d), NAN, dtype=torch.float32, device="cuda")
    lse = torch.full((H, n_seqs * n), NAN, device="cuda")
    lens = torch.full((n_seqs,), length, dtype=torch.int32, device="cuda")
    parents = torch.tensor([x for t in trees for x in t], dtype=torch.int32, device="cuda")
    ws = ralib.new_workspace(ralib.ra_paged_tree_attn_workspace_bytes(n_seqs * n, n_seqs, H, 1, d, n, length, window, 0))
    ralib.ra_paged_tree_attn_fwd(q, k, v, table, lens, cu_of([n] * n_seqs), parents, o, lse, n, length, window, 0, workspace=ws)
    ralib.ra_check_status(ws)
    assert bool(torch.isfinite(o).all())
    kd, vd = k[:, :, 0].double(), v[:, :, 0].double()
    for s in range(0, n_seqs, max(1, n_seqs // 5)):
        for i in range(0, n, max(1, n // 4)):
            path = tr.path(trees[s], i)
            first = max(0, length - n + len(path) - window) if window else 0       # the first place that is seen
            times = torch.zeros((3, page), dtype=torch.float64, device="cuda")
            for p in range(first // page, pages):
                which = 2 if p == pages - 1 else 1 if p >= pages // 2 else 0
                from_ = max(0, first - p * page)
                if p < pages - 1:
                    times[which, from_:] += 1
                else:
                    times[2, from_:page - n] = 1
                    times[2, [page - n + a for a in path]] = 1
            x = torch.einsum("hd,ptd->hpt", q[s * n + i].double(), kd) * d ** -0.5 + times.log()
            le = torch.logsumexp(x.flatten(1), 1)
            w = torch.exp(x - le[:, None, None])
            oe, spread = torch.einsum("hpt,ptd->hd", w, vd), torch.einsum("hpt,ptd->hd", w, vd.abs())
            tol = 2.0 ** -9 * spread + 2.0 ** -8 * (spread + oe.abs()) + 1e-6
            ref.assert_within(o[s * n + i], oe, tol, "sequence %d node %d O" % (s, i))
            # (its sum is rounded at each of a part's 1024 tiles and each of up to 128 parts, 2^-24 of it; EPS for
            # scores of 1.5 times the usual size)
            ref.assert_within(lse[:, s * n + i], le, 1.5 * ref.EPS + 1152 * 2.0 ** -24 + 1e-6 * le.abs(), "sequence %d node %d LSE" % (s, i))


@pytest.mark.parametrize("n_seqs,n,H,d", [(1, 320, 128, 64), (1, 320, 128, 128), (160, 20, 5, 64), (160, 20, 5, 128)])
def test_values_of_one(ralib, gpu, n_seqs, n, H, d):
    """O is 1: what the tensor cores cut off, 2^-9 at most (above), is all that it is off by."""
    page, length = 65536, 1 << 22
    k, v = randn_bf16((2, page, 1, d), 9).cuda(), torch.ones((2, page, 1, d), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((n_seqs, length // page), dtype=torch.int32, device="cuda")
    table[:, -1] = 1
    parents = torch.tensor(tr.random_tree(n, "bush", 2) * n_seqs, dtype=torch.int32, device="cuda")
    q = randn_bf16((n_seqs * n, H, d), 5).cuda()
    o = torch.full((n_seqs * n, H, d), NAN, dtype=torch.float32, device="cuda")
    lens = torch.full((n_seqs,), length, dtype=torch.int32, device="cuda")
    ws = ralib.new_workspace(ralib.ra_paged_tree_attn_workspace_bytes(n_seqs * n, n_seqs, H, 1, d, n, length))
    ralib.ra_paged_tree_attn_fwd(q, k, v, table, lens, cu_of([n] * n_seqs), parents, o, None, n, length, workspace=ws)
    ralib.ra_check_status(ws)
    assert (o - 1).abs().max().item() <= 2.0 ** -9 + 1e-6


@pytest.mark.parametrize("new,lens,H,Hkv,d,page,window,sinks", CASES)
@pytest.mark.parametrize("shape", ["levels", "chain"])
def test_tables_that_could_hold_more(ralib, gpu, new, lens, H, Hkv, d, page, window, sinks, shape):
    """Ordinary contexts in tables for more tokens than are summed in one part."""
    c = Cache(lens, page, Hkv, d, sum(lens) + H)
    c.fill_all()
    c.table = torch.nn.functional.pad(c.table, (0, 140000 // page), value=-1).contiguous()
    q = randn_bf16((sum(new), H, d), 99 + H).cuda()
    trees = trees_of(new, shape)
    o, lse, _ = attend(ralib, c, q, cu_of(new), trees, torch.bfloat16 if shape == "chain" else torch.float32, window, sinks)
    assert_trees(c, q, o, lse, trees, window, sinks)
