"""Timed cases of the operators for speculative decoding over a paged key/value cache: appending new
keys and values with the position rotation applied on the way (queries too), attention of a tree of
drafted tokens over the cache, and keeping the accepted path of the tree in the cache.

``own`` false: the operators in plain torch operations, in 32 bits (the rotation's angles in 64),
rounded once at the end.  ``own`` true: the library's entry points, as a program calls them.

A tree is one int32 per drafted token: the number, among its sequence's drafted tokens, of the token
it follows, or -1 for one that follows the cached context.
"""
import math
import random

import torch

own = False

_NEG = float("-inf")


# ------------------------------------------------------------------ cases
def _tree(name, n, new_min, new_max, len_min, len_max, H, Hkv, d, page, width, W=0, sinks=0, mix=1):
    """len: tokens in the cache, the drafted ones among them; width: nodes of a level of the tree."""
    return {"name": name, "op": "tree", "n": n, "new_min": new_min, "new_max": new_max, "len_min": len_min,
            "len_max": len_max, "H": H, "Hkv": Hkv, "d": d, "page": page, "width": width, "W": W, "sinks": sinks, "mix": mix}


def _append(name, n, new_min, new_max, len_min, len_max, H, Hkv, d, page, rot, pairs=False, width=0, mix=1):
    """rot: rotated columns of a head; pairs: neighbouring columns turn together; width > 0: positions of a tree."""
    return {"name": name, "op": "append", "n": n, "new_min": new_min, "new_max": new_max, "len_min": len_min,
            "len_max": len_max, "H": H, "Hkv": Hkv, "d": d, "page": page, "rot": rot, "pairs": pairs, "width": width, "mix": mix}


def _keep(name, n, layers, new_min, new_max, len_min, len_max, Hkv, d, page, width, mix=1):
    return {"name": name, "op": "keep", "n": n, "layers": layers, "new_min": new_min, "new_max": new_max,
            "len_min": len_min, "len_max": len_max, "Hkv": Hkv, "d": d, "page": page, "width": width, "mix": mix}


def listed():
    return [
        # one conversation, a small draft: the latency of a call
        _tree("tree 8 nodes over 1000", 1, 8, 8, 1000, 1000, 32, 8, 128, 16, 2),
        # one conversation, the usual size of a draft tree, an ordinary context
        _tree("tree 60 nodes over 8K", 1, 60, 60, 8192, 8192, 32, 8, 128, 64, 10),
        # a long document, 16 drafted tokens: the cache's bytes
        _tree("tree 16 nodes over 128K", 1, 16, 16, 131072, 131072, 32, 8, 128, 128, 4),
        # a serving batch with trees and contexts of different sizes
        _tree("tree batch 32", 32, 8, 26, 200, 8000, 32, 8, 128, 64, 5),
        # a large batch with few drafted tokens each
        _tree("tree batch 64 small", 64, 4, 8, 500, 12000, 32, 8, 128, 16, 2),
        # streaming decode: long contexts of which a window and the sinks are read
        _tree("tree window 64K", 8, 40, 40, 60000, 65536, 16, 2, 64, 128, 8, W=4096, sinks=4),
        # offline drafting with wide trees, the most nodes
        _tree("tree 500 nodes", 2, 300, 500, 4000, 16000, 16, 4, 64, 32, 40),
        # the new token of each of 64 conversations, before single-token attention
        _append("append rotary 64 tokens", 64, 1, 1, 1, 4000, 32, 8, 128, 16, 128),
        # three prompts whole
        _append("append rotary prompts", 3, 5000, 8000, 8000, 9000, 32, 8, 128, 64, 128),
        # the drafted trees of 16 conversations far into long contexts, a part of the columns rotated in neighbouring pairs
        _append("append rotary trees", 16, 26, 60, 60000, 131072, 16, 4, 64, 256, 32, pairs=True, width=8),
        # one conversation's accepted path, the cache of a few layers
        _keep("keep path one", 1, 4, 26, 26, 1000, 1000, 8, 128, 16, 8),
        # a serving batch, the caches of 16 layers in one pool
        _keep("keep path batch 48", 48, 16, 20, 60, 100, 600, 8, 128, 16, 10),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "append", "append", "keep"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 4, 5, 8])
    mix = rng.randrange(1 << 20)
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "tree":
        new_max = rng.choice([_log_int(rng, 1, 8), _log_int(rng, 8, 64), _log_int(rng, 8, 64), _log_int(rng, 64, 500)])
        len_max = new_max + _log_int(rng, 1, 131072 - 500)
        n = _log_int(rng, 1, 64)
        # no more than the largest listed cases' cache, and scores that the plain form can hold
        while n > 1 and (n * len_max * Hkv * d > 64 * 6000 * 8 * 128 or n * len_max * new_max * H > 2 * 16000 * 500 * 16):
            n = (n + 1) // 2
        while new_max > 1 and len_max * new_max * H > 2 * 16000 * 500 * 16:
            new_max = (new_max + 1) // 2
        W = rng.choice([0, 0, _log_int(rng, 1, 4096)])
        return {"op": op, "n": n, "new_min": rng.choice([0, 1, (new_max + 1) // 2]), "new_max": new_max, "len_min": new_max,
                "len_max": len_max, "H": H, "Hkv": Hkv, "d": d, "page": page, "width": _log_int(rng, 1, 40), "W": W,
                "sinks": rng.choice([0, 4, 130]) if W else 0, "mix": mix}
    if op == "append":
        tree = rng.random() < 0.4
        new_max = _log_int(rng, 1, 64) if tree else rng.choice([1, _log_int(rng, 1, 8000)])
        n = _log_int(rng, 1, 64 if new_max < 200 else 3)
        len_max = new_max + _log_int(rng, 1, 131072 if n * Hkv * d <= 16 * 4 * 64 else 4000)
        return {"op": op, "n": n, "new_min": (new_max + 1) // 2, "new_max": new_max, "len_min": new_max, "len_max": len_max,
                "H": H, "Hkv": Hkv, "d": d, "page": page, "rot": rng.choice([16, 32, 48, 64] + ([96, 128, 128] if d == 128 else [64])),
                "pairs": rng.random() < 0.4, "width": rng.randint(1, 10) if tree else 0, "mix": mix}
    new_max = _log_int(rng, 1, 200)
    return {"op": op, "n": _log_int(rng, 1, 48), "layers": _log_int(rng, 1, 16), "new_min": (new_max + 1) // 2, "new_max": new_max,
            "len_min": new_max, "len_max": new_max + _log_int(rng, 1, 500), "Hkv": Hkv, "d": d, "page": page,
            "width": rng.randint(1, 12), "mix": mix}


def _lens(case):
    """Each sequence's new tokens and its tokens in the cache, the new ones among them."""
    r = random.Random(case["mix"])
    new = [r.randint(case["new_min"], case["new_max"]) for _ in range(case["n"])]
    new[0] = case["new_max"]
    total = [max(k, r.randint(case["len_min"], case["len_max"])) for k in new]
    return new, total


def _parents(case):
    """Each sequence's tree: node 0, then levels of `width` nodes, each under some node of the level before."""
    new, _ = _lens(case)
    r = random.Random(case["mix"] + 1)
    w = case["width"]
    trees = []
    for n in new:
        level = [0] + [1 + (i - 1) // w for i in range(1, n)]
        first = lambda k: 0 if k == 0 else 1 + (k - 1) * w      # noqa: E731
        trees.append([-1] + [r.randrange(first(level[i] - 1), first(level[i])) for i in range(1, n)] if n else [])
    return trees


def _accepted(case):
    """The trees, and each sequence's last accepted node (-1: none).  A pass moves tokens inside the pool, and a second
    one on the same state has to find the same, so the node's path is one whose moved nodes all lie behind the path's
    length: their places are read and not written."""
    trees = _parents(case)
    r = random.Random(case["mix"] + 2)
    last = []
    for p in trees:
        fit = [-1]
        for i in range(len(p)):
            path = _path(p, i)
            if all(a == j or a >= len(path) for j, a in enumerate(path)):
                fit.append(i)
        deep = sorted(fit, key=lambda i: len(_path(p, i)))
        last.append(r.choice(deep[len(deep) // 2:]))        # drafts are mostly accepted to some depth
    return trees, last


def _path(p, i):
    path = []
    while i >= 0:
        path.append(i)
        i = p[i]
    return path[::-1]


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _flat(trees):
    return _ints([x for p in trees for x in p])


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    n, page, Hkv, d = case["n"], case["page"], case["Hkv"], case["d"]
    new, total = _lens(case)
    # a cache: pages in no order, a table of each sequence's pages
    held = [-(-t // page) for t in total]
    n_pages = sum(held) + 3
    order = torch.randperm(n_pages, generator=_gen(seed + 1), device="cuda").to(torch.int32)
    width = max(held)
    col = torch.arange(width, device="cuda")
    first = torch.tensor([0] + held[:-1], device="cuda").cumsum(0)
    has = col[None, :] < torch.tensor(held, device="cuda")[:, None]
    at = (first[:, None] + col[None, :]).clamp(max=n_pages - 1)
    s["table"] = torch.where(has, order[at], torch.full_like(order[at], -1)).contiguous()
    s["seq_lens"], s["new"], s["total"] = _ints(total), new, total
    s["cu"] = torch.cat([_ints([0]), _ints(new).cumsum(0).to(torch.int32)])
    s["T"] = T = sum(new)
    pool = (n_pages, page, Hkv, d) if case["op"] != "keep" else (case["layers"], n_pages, page, Hkv, d)
    s["k_pages"], s["v_pages"] = _randn(g, *pool), _randn(g, *pool)
    if case["op"] == "keep":
        trees, last = _accepted(case)
        s["parents"], s["last"] = _flat(trees), _ints(last)
        s["new_lens"], s["path"] = torch.empty_like(s["seq_lens"]), torch.empty_like(s["parents"])
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        return s
    H = case["H"]
    s["parents"] = _flat(_parents(case)) if case["width"] else None
    if case["op"] == "append":
        # a layer's fused projection: queries, keys and values of a token beside one another
        s["qkv"] = _randn(g, T, H + 2 * Hkv, d)
        s["q"], s["k_new"], s["v_new"] = s["qkv"][:, :H], s["qkv"][:, H:H + Hkv], s["qkv"][:, H + Hkv:]
        s["q_out"] = torch.empty((T, H, d), dtype=torch.bfloat16, device="cuda")
        half = case["rot"] // 2
        s["inv_freq"] = (500000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        return s
    s["q"] = _randn(g, T, H, d)
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((H, T), dtype=torch.float32, device="cuda")
    # partial results of a context split over the key axis: at most this many bytes
    s["ws"] = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _rows(s):
    """Each new token's sequence and number in it."""
    cu = s["cu"].long()
    t = torch.arange(s["T"], device=cu.device)
    seq = torch.bucketize(t, cu[1:], right=True)
    return seq, t - cu[seq]


def _ancestors(s, most):
    """[n, most, most]: whether node j is i or one of its ancestors."""
    seq, i = _rows(s)
    a = torch.zeros((s["n"], most, most), device="cuda")
    a[seq, i, i] = 1
    p = s["parents"].long()
    a[seq[p >= 0], i[p >= 0], p[p >= 0]] = 1
    k = 1
    while k < most:
        a = (a @ a > 0).float()
        k *= 2
    return a > 0


def _tree_plain(s):
    n, Hkv, d, page, H = s["n"], s["Hkv"], s["d"], s["page"], s["H"]
    G, most = H // Hkv, max(s["new"])
    table = s["table"].long().clamp(min=0)
    M = table.shape[1] * page
    lens = s["seq_lens"].long()
    at = torch.arange(M, device="cuda")
    written = (at[None, :] < lens[:, None]).reshape(n, M, 1, 1)
    kk, vv = (torch.where(written, x[table].reshape(n, M, Hkv, d), 0).float().permute(0, 2, 1, 3)
              for x in (s["k_pages"], s["v_pages"]))
    cu = s["cu"].long()
    count = cu[1:] - cu[:-1]
    c = lens - count
    i = torch.arange(most, device="cuda")
    inside = i[None, :] < count[:, None]
    q = s["q"][(cu[:-1, None] + i).clamp(max=s["T"] - 1)].float()                       # [n, most, H, d]
    q = q.reshape(n, most, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(n, Hkv, most * G, d)
    anc = _ancestors(s, most)
    depth = anc.sum(-1) - 1                                                            # [n, most]
    pos = c[:, None] + depth
    j = at[None, :] - c[:, None]                                                       # [n, M]
    drafted = (j >= 0) & (j < count[:, None])
    jc = j.clamp(0, most - 1)
    seen = torch.gather(anc, 2, jc[:, None, :].expand(n, most, M)) & drafted[:, None, :]
    seen |= (j < 0)[:, None, :]
    if s["W"]:
        kp = torch.where(j < 0, at[None, :].expand(n, M), c[:, None] + torch.gather(depth, 1, jc))[:, None, :]
        seen &= (kp > pos[..., None] - s["W"]) | (kp < s["sinks"])
    x = q @ kk.transpose(-1, -2) * (1.0 / math.sqrt(d))
    x = x.masked_fill_(~seen.repeat_interleave(G, 1)[:, None], _NEG)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == _NEG, torch.zeros_like(m), m))
    t = p.sum(-1, keepdim=True)
    o = (p @ vv) / t
    lse = (m + torch.log(t))[..., 0]
    o = o.reshape(n, Hkv, most, G, d).permute(0, 2, 1, 3, 4).reshape(n, most, H, d)[inside]
    lse = lse.reshape(n, Hkv, most, G).permute(0, 2, 1, 3).reshape(n, most, H)[inside]
    return o.to(torch.bfloat16), lse.t().contiguous()


def _rotated(x, cos, sin, rot, pairs):
    """x [T, heads, d] with its first `rot` columns turned, in bf16."""
    y = x.float()
    if pairs:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
    else:
        a, b = y[..., : rot // 2], y[..., rot // 2: rot]
    c, si = cos[:, None], sin[:, None]
    a, b = a * c - b * si, a * si + b * c
    turned = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(torch.bfloat16)


def _append_plain(s):
    seq, i = _rows(s)
    cu = s["cu"].long()
    c = s["seq_lens"].long()[seq] - (cu[seq + 1] - cu[seq])
    slot = c + i
    pos = slot if s["parents"] is None else c + (_ancestors(s, max(s["new"])).sum(-1) - 1)[seq, i]
    angle = pos.double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    page = s["table"][seq, slot // s["page"]].long()
    s["k_pages"][page, slot % s["page"]] = _rotated(s["k_new"], cos, sin, s["rot"], s["pairs"])
    s["v_pages"][page, slot % s["page"]] = s["v_new"]
    return _rotated(s["q"], cos, sin, s["rot"], s["pairs"]), s["k_pages"], s["v_pages"]


def _keep_plain(s):
    most = max(s["new"])
    cu = s["cu"].long()
    count = cu[1:] - cu[:-1]
    c = s["seq_lens"].long() - count
    anc = _ancestors(s, most)
    last = s["last"].long()
    on = torch.gather(anc, 1, last.clamp(min=0)[:, None, None].expand(-1, 1, most))[:, 0] & (last >= 0)[:, None]
    j = on.long().cumsum(1) - 1                                     # a node's place on the path
    seq, node = on.nonzero(as_tuple=True)
    to = j[seq, node]
    page = s["page"]
    here, there = c[seq] + node, c[seq] + to
    fp, tp = s["table"][seq, here // page].long(), s["table"][seq, there // page].long()
    for x in (s["k_pages"], s["v_pages"]):
        x[:, tp, there % page] = x[:, fp, here % page]
    path = torch.full_like(s["path"], -1)
    path[cu[seq] + to] = (cu[seq] + node).to(torch.int32)
    return s["k_pages"], s["v_pages"], (c + on.sum(1)).to(torch.int32), path


# ------------------------------------------------------------------ the pass
def run(s):
    op = s["op"]
    if not own:
        return {"tree": _tree_plain, "append": _append_plain, "keep": _keep_plain}[op](s)
    import sequence_blockwise_softmax_gb300 as ra

    if op == "tree":
        ra.ra_paged_tree_attn_fwd(s["q"], s["k_pages"], s["v_pages"], s["table"], s["seq_lens"], s["cu"], s["parents"],
                                  s["o"], s["lse"], max_new=s["new_max"], max_len=s["len_max"], window=s["W"],
                                  sinks=s["sinks"], workspace=s["ws"])
        return s["o"], s["lse"]
    if op == "append":
        ra.ra_paged_append_rotary(s["q"], s["k_new"], s["v_new"], s["q_out"], s["k_pages"], s["v_pages"], s["table"],
                                  s["seq_lens"], s["cu"], s["inv_freq"], parents=s["parents"], pairs=s["pairs"],
                                  workspace=s["ws"])
        return s["q_out"], s["k_pages"], s["v_pages"]
    ra.ra_paged_keep_path(s["k_pages"], s["v_pages"], s["table"], s["seq_lens"], s["cu"], s["parents"], s["last"],
                          s["new_lens"], s["path"], workspace=s["ws"])
    return s["k_pages"], s["v_pages"], s["new_lens"], s["path"]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    new, total = _lens(case)
    T, token = sum(new), case["Hkv"] * case["d"] * 2
    if case["op"] == "append":
        return {"bytes": 2 * T * (case["H"] * case["d"] * 2 + 2 * token), "flops": 3 * T * (case["H"] + case["Hkv"]) * case["rot"]}
    if case["op"] == "keep":
        trees, last = _accepted(case)
        moved = sum(a != j for p, i in zip(trees, last) for j, a in enumerate(_path(p, i)))
        return {"bytes": 4 * moved * token * case["layers"] + 8 * T + 12 * case["n"], "flops": 0}
    W, sinks = case["W"], case["sinks"]
    pairs = read = 0
    for p, n, t in zip(_parents(case), new, total):
        c = t - n
        depth = []
        for x in p:
            depth.append(depth[x] + 1 if x >= 0 else 0)
        for e in depth:
            near = min(c + e + 1, W) if W else c + e + 1
            pairs += near + min(sinks, c + e + 1 - near)
        read += n + (min(c, max(0, W - 1) + sinks) if W else c) if n else 0
    rows = T * case["H"]
    return {"bytes": 2 * read * token + rows * (4 * case["d"] + 4) + 4 * T, "flops": 4 * case["d"] * pairs * case["H"]}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_tree(case, s):
    H, Hkv, d, page, W = case["H"], case["Hkv"], case["d"], case["page"], case["W"]
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty((H, s["T"]), dtype=torch.float64, device="cuda")
    t0 = 0
    for i, (p, n, total) in enumerate(zip(_parents(case), s["new"], s["total"])):
        if not n:
            continue
        c = total - n
        paths = [_path(p, x) for x in range(n)]
        lo = max(0, c - W + 1) if W else 0
        # the slots that some row may see, and their positions
        slots = list(range(min(case["sinks"], lo))) + list(range(lo, total)) if W else list(range(total))
        at = torch.tensor(slots, device="cuda")
        kpos = torch.tensor([x if x < c else c + len(paths[x - c]) - 1 for x in slots], device="cuda")
        where = {x: y for y, x in enumerate(slots)}
        ok = torch.zeros((n, len(slots)), dtype=torch.bool)
        ok[:, : len(slots) - n] = True
        for x, path in enumerate(paths):
            ok[x, [where[c + y] for y in path]] = True
        ok = ok.cuda()
        pos = torch.tensor([c + len(x) - 1 for x in paths], device="cuda")
        if W:
            ok &= (kpos[None, :] > pos[:, None] - W) | (kpos[None, :] < case["sinks"])
        pages = s["table"][i, : -(-total // page)].long()
        k, v = (x[pages].reshape(-1, Hkv, d)[at].permute(1, 0, 2).double() for x in (s["k_pages"], s["v_pages"]))
        step = max(1, (1 << 27) // (H * len(slots)))
        for r0 in range(0, n, step):
            r1 = min(n, r0 + step)
            q = s["q"][t0 + r0: t0 + r1].double().permute(1, 0, 2).reshape(Hkv, -1, d)      # group by rows
            x = torch.einsum("hrd,htd->hrt", q, k) / math.sqrt(d)
            x = x.reshape(H, r1 - r0, -1)
            x[:, ~ok[r0:r1]] = _NEG
            ll = torch.logsumexp(x, -1)
            w = torch.exp(x - ll[..., None])
            oo = torch.einsum("hrt,htd->hrd", w.reshape(Hkv, -1, w.shape[2]), v).reshape(H, r1 - r0, d)
            o[t0 + r0: t0 + r1], lse[:, t0 + r0: t0 + r1] = oo.permute(1, 0, 2), ll
        t0 += n
    return o, lse


def _exact_append(case, s):
    rot = case["rot"]
    trees = _parents(case) if case["width"] else None
    pos, page_of, off = [], [], []
    table = s["table"].tolist()
    for i, (n, total) in enumerate(zip(s["new"], s["total"])):
        for x in range(n):
            slot = total - n + x
            pos.append(slot if trees is None else total - n + len(_path(trees[i], x)) - 1)
            page_of.append(table[i][slot // case["page"]])
            off.append(slot % case["page"])
    pos = torch.tensor(pos, dtype=torch.float64, device="cuda")

    def turn(x):
        y = x.double().clone()
        for m in range(rot // 2):
            a, b = (2 * m, 2 * m + 1) if case["pairs"] else (m, m + rot // 2)
            phi = (pos * s["inv_freq"][m].double())[:, None]
            xa, xb = x[..., a].double(), x[..., b].double()
            y[..., a], y[..., b] = xa * phi.cos() - xb * phi.sin(), xa * phi.sin() + xb * phi.cos()
        return y

    k, v = s["k_pages"].double(), s["v_pages"].double()
    at = torch.tensor(page_of, device="cuda"), torch.tensor(off, device="cuda")
    k[at], v[at] = turn(s["k_new"]), s["v_new"].double()
    return turn(s["q"]), k, v


def _exact_keep(case, s):
    k, v = s["k_pages"].double(), s["v_pages"].double()
    trees, last = _accepted(case)
    table = s["table"].tolist()
    lens, rows, first = [], [], 0
    for i, (p, leaf, total) in enumerate(zip(trees, last, s["total"])):
        path, c = _path(p, leaf), total - len(p)
        for j, a in enumerate(path):      # ascending: a node's place is read before a later one lands there
            src, dst = c + a, c + j
            for x in (k, v):
                x[:, table[i][dst // case["page"]], dst % case["page"]] = x[:, table[i][src // case["page"]], src % case["page"]].clone()
        lens.append(c + len(path))
        rows += [first + a for a in path] + [-1] * (len(p) - len(path))
        first += len(p)
    return k, v, _ints(lens), _ints(rows)


def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "append": _exact_append, "keep": _exact_keep}[case["op"]](case, s)
