"""Timed cases of the attention operators for long contexts: sliding-window attention with
sinks (forward and backward), attention of new tokens over a paged key/value cache (single
tokens and chunks), and appending new keys and values to that cache.

``own`` false: the operators in plain torch operations, in 32 bits, rounded once at the end.
``own`` true: the library's entry points, as a program calls them.
"""
import math
import random

import torch

own = False

_NEG = float("-inf")


# ------------------------------------------------------------------ cases
def _window(name, op, B, L, H, Hkv, d, W, sinks, n_seqs=0, mix=1):
    return {"name": name, "op": op, "B": B, "L": L, "H": H, "Hkv": Hkv, "d": d, "W": W, "sinks": sinks,
            "n_seqs": n_seqs, "mix": mix}


def _paged(name, n, new_min, new_max, len_min, len_max, H, Hkv, d, page, W=0, sinks=0, mix=1):
    return {"name": name, "op": "paged", "n": n, "new_min": new_min, "new_max": new_max, "len_min": len_min,
            "len_max": len_max, "H": H, "Hkv": Hkv, "d": d, "page": page, "W": W, "sinks": sinks, "mix": mix}


def _append(name, n, new_min, new_max, len_min, len_max, Hkv, d, page, mix=1):
    return {"name": name, "op": "append", "n": n, "new_min": new_min, "new_max": new_max, "len_min": len_min,
            "len_max": len_max, "Hkv": Hkv, "d": d, "page": page, "mix": mix}


def listed():
    return [
        # one short prompt of a small model: the launch's own cost
        _window("window fwd 512", "window_fwd", 1, 512, 2, 2, 64, 128, 4),
        # a training or prefill pass over 8K tokens, window 1024
        _window("window fwd 8K", "window_fwd", 1, 8192, 16, 16, 128, 1024, 4),
        # a 128K document, the longest prefill here
        _window("window fwd 128K", "window_fwd", 1, 131072, 8, 8, 128, 1024, 64),
        # a packed training batch of five documents, odd length, shared key/value heads
        _window("window bwd packed", "window_bwd", 1, 8191, 16, 4, 64, 500, 3, n_seqs=5),
        # the gradient of a 32K training sequence with a wide window
        _window("window bwd 32K", "window_bwd", 1, 32768, 8, 8, 128, 2048, 128),
        # one conversation answering token by token
        _paged("decode one", 1, 1, 1, 1000, 1000, 32, 8, 128, 16),
        # a serving batch of 64 conversations of very different lengths
        _paged("decode 64 ragged", 64, 1, 1, 200, 16000, 32, 8, 128, 64),
        # streaming decode: contexts of 128K of which a window and four sinks are read
        _paged("decode window 128K", 16, 1, 1, 100000, 131072, 16, 2, 64, 128, W=4096, sinks=4),
        # a chunk of a long prompt over what the cache already holds
        _paged("chunk 512 over 32K", 1, 512, 512, 32768, 32768, 32, 8, 128, 16),
        # chunked prefill and decoding mixed in one batch
        _paged("mixed chunks", 8, 1, 700, 700, 9000, 16, 4, 64, 32),
        # the new token of each of 64 conversations goes into the cache
        _append("append 64 tokens", 64, 1, 1, 1, 4000, 8, 128, 16),
        # three prompts go into the cache whole
        _append("append prompts", 3, 5000, 8000, 8000, 9000, 8, 128, 64),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window_fwd", "window_fwd", "window_bwd", "paged", "paged", "paged", "append"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    mix = rng.randrange(1 << 20)
    if op in ("window_fwd", "window_bwd"):
        H = Hkv * rng.choice([1, 2, 3, 4])
        B = rng.choice([1, 1, 2])
        L = _log_int(rng, 1, 131072 if op == "window_fwd" else 32768)
        W = _log_int(rng, 1, 4096)
        # at most the largest listed case's products, whose scores the plain form holds
        most = 8 * 131072 * 1024 if op == "window_fwd" else 8 * 32768 * 2048
        while B * H * L * min(L, max(W, 64)) > most // 2:
            L = (L + 1) // 2
        n_seqs = 0
        if B == 1 and rng.random() < 0.4:
            L = max(1, L // 4)
            n_seqs = _log_int(rng, 1, min(L, 12))
        return {"op": op, "B": B, "L": L, "H": H, "Hkv": Hkv, "d": d, "W": W,
                "sinks": rng.choice([0, 1, 4, 100, 129]), "n_seqs": n_seqs, "mix": mix}
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        new_max = _log_int(rng, 1, 4000)
        len_max = new_max + _log_int(rng, 1, 4000)
        return {"op": op, "n": _log_int(rng, 1, 64 if new_max < 200 else 4), "new_min": (new_max + 1) // 2, "new_max": new_max,
                "len_min": new_max, "len_max": len_max, "Hkv": Hkv, "d": d, "page": page, "mix": mix}
    H = Hkv * rng.choice([1, 2, 4, 5, 8])
    new_max = rng.choice([1, 1, rng.randrange(2, 9), _log_int(rng, 9, 600)])
    len_max = new_max + _log_int(rng, 1, 32768)
    n = _log_int(rng, 1, 64)
    while n > 1 and (n * len_max * Hkv * d > 32 * 16000 * 8 * 128 or n * len_max * new_max * H > 32768 * 512 * 32):
        n = (n + 1) // 2
    while new_max > 1 and len_max * new_max * H > 32768 * 512 * 32:
        new_max = (new_max + 1) // 2
    W = rng.choice([0, 0, _log_int(rng, 1, 4096)])
    return {"op": op, "n": n, "new_min": 1, "new_max": new_max, "len_min": new_max, "len_max": len_max, "H": H,
            "Hkv": Hkv, "d": d, "page": page, "W": W, "sinks": rng.choice([0, 4, 130]) if W else 0, "mix": mix}


def _lens(case):
    """The lengths a case stands for: of its packed sequences (they add up to L), or (new tokens, cache lengths)."""
    r = random.Random(case["mix"])
    if "n" in case:
        new = [r.randint(case["new_min"], case["new_max"]) for _ in range(case["n"])]
        new[0] = case["new_max"]
        total = [max(k, r.randint(case["len_min"], case["len_max"])) for k in new]
        return new, total
    if not case["n_seqs"]:
        return [case["L"]] * case["B"]
    cuts = sorted(r.sample(range(1, case["L"]), case["n_seqs"] - 1)) if case["n_seqs"] > 1 else []
    edges = [0] + cuts + [case["L"]]
    return [b - a for a, b in zip(edges, edges[1:])]


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _edges(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def _new_workspace(nbytes):
    return torch.zeros((max(256, int(nbytes)) + 15) // 16 * 16, dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] in ("window_fwd", "window_bwd"):
        B, L, H, Hkv, d = (case[k] for k in ("B", "L", "H", "Hkv", "d"))
        s["lens"] = _lens(case)
        s["q"], s["k"], s["v"] = _randn(g, B, L, H, d), _randn(g, B, L, Hkv, d), _randn(g, B, L, Hkv, d)
        s["cu"] = _edges(s["lens"]) if case["n_seqs"] else None
        s["o"] = torch.empty((B, L, H, d), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((B, H, L), dtype=torch.float32, device="cuda")
        if case["op"] == "window_bwd":
            s["do"] = _randn(g, B, L, H, d)
            o, lse = _window_fwd_plain(s)       # what the forward left behind
            s["o"].copy_(o)
            s["lse"].copy_(lse)
            s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[x]) for x in ("q", "k", "v"))
            # the sums over a row, and the sinks' partial gradients from each chunk of queries
            s["ws"] = _new_workspace(4 * B * L * H + (64 << 20))
        else:
            s["ws"] = _new_workspace(256)
        return s
    # a cache: pages in no order, a table of each sequence's pages, what lies behind the last token never written
    n, page, Hkv, d = case["n"], case["page"], case["Hkv"], case["d"]
    new, total = _lens(case)
    held = [-(-t // page) for t in total]
    n_pages = sum(held) + 3
    order = torch.randperm(n_pages, generator=_gen(seed + 1), device="cuda").to(torch.int32)
    width = max(held)
    col = torch.arange(width, device="cuda")
    first = torch.tensor([0] + held[:-1], device="cuda").cumsum(0)
    has = col[None, :] < torch.tensor(held, device="cuda")[:, None]
    at = (first[:, None] + col[None, :]).clamp(max=n_pages - 1)
    s["table"] = torch.where(has, order[at], torch.full_like(order[at], -1)).contiguous()
    s["seq_lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    s["new"], s["total"], s["cu"] = new, total, _edges(new)
    s["T"] = sum(new)
    s["k_pages"], s["v_pages"] = _randn(g, n_pages, page, Hkv, d), _randn(g, n_pages, page, Hkv, d)
    if case["op"] == "append":
        s["k_new"], s["v_new"] = _randn(g, s["T"], Hkv, d), _randn(g, s["T"], Hkv, d)
        s["ws"] = _new_workspace(256)
        return s
    s["q"] = _randn(g, s["T"], case["H"], d)
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((case["H"], s["T"]), dtype=torch.float32, device="cuda")
    # partial results of a context split over the key axis: at most this many rows
    s["ws"] = _new_workspace(64 << 20)
    return s


# ------------------------------------------------------------------ plain forms
def _padded(x, lens, cu):
    """[B, L, ...] (or one packed run of sequences) as [n, longest, ...] in 32 bits, zeros behind each end."""
    if cu is None:
        return x.float()
    start = cu[:-1].long()
    at = start[:, None] + torch.arange(max(lens), device=x.device)
    inside = at < cu[1:].long()[:, None]
    y = x[0][at.clamp(max=x.shape[1] - 1)].float()
    return y * inside.reshape(inside.shape + (1,) * (y.dim() - 2))


def _unpadded(y, lens, cu):
    """The inverse of _padded."""
    if cu is None:
        return y
    M = y.shape[1]
    inside = torch.arange(M, device=y.device)[None, :] < (cu[1:] - cu[:-1]).long()[:, None]
    return y[inside][None]


class _Band:
    """The pairs of a windowed attention in blocks of C >= W queries: block i meets the keys of blocks
    i - 1 and i, and the sinks those leave out."""

    def __init__(self, s, n, M):
        W = max(1, min(s["W"], M))
        self.C = C = max(W, min(M, 64))
        self.nb, self.M, self.n = -(-M // C), M, n
        self.ns = min(s["sinks"], M)
        self.Hkv, self.G, self.d = s["Hkv"], s["H"] // s["Hkv"], s["d"]
        dev = s["q"].device
        qp = torch.arange(self.nb * C, device=dev).reshape(self.nb, C, 1)
        kp = (torch.arange(self.nb, device=dev) * C - C).reshape(-1, 1, 1) + torch.arange(2 * C, device=dev)
        near = (kp >= 0) & (kp <= qp) & (kp > qp - W)
        sk = torch.arange(self.ns, device=dev).reshape(1, 1, -1)
        self.seen = torch.cat([near, (sk <= qp - W).expand(self.nb, C, self.ns)], -1)   # [nb, C, 2C + ns]

    def blocks(self, x):
        """[n, M, h, d] as [n, h, nb, C, d]."""
        n, M, h, d = x.shape
        x = torch.cat([x, x.new_zeros(n, self.nb * self.C - M, h, d)], 1)
        return x.reshape(n, self.nb, self.C, h, d).permute(0, 3, 1, 2, 4)

    def queries(self, x):
        """[n, M, H, e] as [n, Hkv, nb, G * C, e]."""
        e = x.shape[-1]
        b = self.blocks(x).reshape(self.n, self.Hkv, self.G, self.nb, self.C, e)
        return b.permute(0, 1, 3, 2, 4, 5).reshape(self.n, self.Hkv, self.nb, self.G * self.C, e)

    def from_queries(self, b):
        e = b.shape[-1]
        b = b.reshape(self.n, self.Hkv, self.nb, self.G, self.C, e).permute(0, 2, 4, 1, 3, 5)
        return b.reshape(self.n, self.nb * self.C, self.Hkv * self.G, e)[:, : self.M]

    def keys(self, x):
        """[n, M, Hkv, d] as each block's [n, Hkv, nb, 2C + ns, d]."""
        b = self.blocks(x)
        prev = torch.cat([torch.zeros_like(b[:, :, :1]), b[:, :, :-1]], 2)
        sink = x[:, : self.ns].permute(0, 2, 1, 3)[:, :, None].expand(-1, -1, self.nb, -1, -1)
        return torch.cat([prev, b, sink], 3)

    def from_keys(self, g):
        """The gradient of keys(): each key's sum over the blocks that met it."""
        C = self.C
        prev, this, sink = g[..., :C, :], g[..., C: 2 * C, :], g[..., 2 * C:, :]
        b = this + torch.cat([prev[:, :, 1:], torch.zeros_like(prev[:, :, :1])], 2)
        x = b.permute(0, 2, 3, 1, 4).reshape(self.n, self.nb * C, self.Hkv, self.d)[:, : self.M].clone()
        x[:, : self.ns] += sink.sum(2).permute(0, 2, 1, 3)
        return x

    def scores(self, s, q, k):
        x = q @ k.transpose(-1, -2) * (1.0 / math.sqrt(self.d))
        seen = self.seen.repeat(1, self.G, 1)
        return x.masked_fill_(~seen, _NEG)


def _softmax_parts(x):
    """exp(x - max), its sum and the log of the sum of exponentials, along the last axis; rows of nothing give 0 and -inf."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == _NEG, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    t = p.sum(-1, keepdim=True)
    return p, t, (m + torch.log(t))[..., 0]


def _window_fwd_plain(s):
    q, k, v = (_padded(s[x], s["lens"], s["cu"]) for x in ("q", "k", "v"))
    band = _Band(s, q.shape[0], q.shape[1])
    p, t, lse = _softmax_parts(band.scores(s, band.queries(q), band.keys(k)))
    o = (p @ band.keys(v)) / torch.where(t == 0, torch.ones_like(t), t)
    o = _unpadded(band.from_queries(o), s["lens"], s["cu"])
    lse = _unpadded(band.from_queries(lse[..., None]), s["lens"], s["cu"])[..., 0]
    return o.to(torch.bfloat16), lse.transpose(1, 2).contiguous()


def _window_bwd_plain(s):
    q, k, v, do, o = (_padded(s[x], s["lens"], s["cu"]) for x in ("q", "k", "v", "do", "o"))
    lse = _padded(s["lse"].transpose(1, 2)[..., None], s["lens"], s["cu"])
    band = _Band(s, q.shape[0], q.shape[1])
    qb, kb, vb, dob = band.queries(q), band.keys(k), band.keys(v), band.queries(do)
    p = torch.exp(band.scores(s, qb, kb) - band.queries(lse))
    dv = band.from_keys(p.transpose(-1, -2) @ dob)
    ds = p * (dob @ vb.transpose(-1, -2) - band.queries((do * o).sum(-1, keepdim=True)))
    scale = 1.0 / math.sqrt(band.d)
    dq = band.from_queries(ds @ kb) * scale
    dk = band.from_keys(ds.transpose(-1, -2) @ qb) * scale
    return tuple(_unpadded(x, s["lens"], s["cu"]).to(torch.bfloat16) for x in (dq, dk, dv))


def _paged_plain(s):
    n, Hkv, d, page, H = s["n"], s["Hkv"], s["d"], s["page"], s["H"]
    G, most = H // Hkv, max(s["new"])
    table = s["table"].long().clamp(min=0)
    M = table.shape[1] * page
    lens = s["seq_lens"].long()
    at = torch.arange(M, device=table.device)
    written = (at[None, :] < lens[:, None]).reshape(n, M, 1, 1)
    kk, vv = (torch.where(written, x[table].reshape(n, M, Hkv, d), 0).float().permute(0, 2, 1, 3)
              for x in (s["k_pages"], s["v_pages"]))
    cu = s["cu"].long()
    count = cu[1:] - cu[:-1]
    i = torch.arange(most, device=table.device)
    inside = i[None, :] < count[:, None]
    q = s["q"][(cu[:-1, None] + i).clamp(max=s["T"] - 1)].float()                       # [n, most, H, d]
    q = q.reshape(n, most, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(n, Hkv, most * G, d)
    pos = (lens - count)[:, None] + i                                                  # [n, most]
    seen = at <= pos[..., None]
    if s["W"]:
        seen = seen & ((at > pos[..., None] - s["W"]) | (at < s["sinks"]))
    x = q @ kk.transpose(-1, -2) * (1.0 / math.sqrt(d))
    x = x.masked_fill_(~seen.repeat_interleave(G, 1)[:, None], _NEG)
    p, t, lse = _softmax_parts(x)
    o = (p @ vv) / t
    o = o.reshape(n, Hkv, most, G, d).permute(0, 2, 1, 3, 4).reshape(n, most, H, d)[inside]
    lse = lse.reshape(n, Hkv, most, G).permute(0, 2, 1, 3).reshape(n, most, H)[inside]
    return o.to(torch.bfloat16), lse.t().contiguous()


def _append_plain(s):
    cu, lens = s["cu"].long(), s["seq_lens"].long()
    t = torch.arange(s["T"], device=cu.device)
    seq = torch.bucketize(t, cu[1:], right=True)
    pos = lens[seq] - (cu[seq + 1] - t)
    page = s["table"][seq, pos // s["page"]].long()
    s["k_pages"][page, pos % s["page"]] = s["k_new"]
    s["v_pages"][page, pos % s["page"]] = s["v_new"]
    return s["k_pages"], s["v_pages"]


# ------------------------------------------------------------------ the pass
def run(s):
    op = s["op"]
    if not own:
        return {"window_fwd": _window_fwd_plain, "window_bwd": _window_bwd_plain, "paged": _paged_plain,
                "append": _append_plain}[op](s)
    import sequence_blockwise_softmax_gb300 as ra

    if op == "window_fwd":
        ra.ra_window_attn_fwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["B"], s["L"], s["H"], s["Hkv"], s["d"],
                              s["W"], s["sinks"], cu_seqlens=s["cu"], workspace=s["ws"])
        return s["o"], s["lse"]
    if op == "window_bwd":
        ra.ra_window_attn_bwd(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], s["dq"], s["dk"], s["dv"], s["B"],
                              s["L"], s["H"], s["Hkv"], s["d"], s["W"], s["sinks"], cu_seqlens=s["cu"],
                              workspace=s["ws"])
        return s["dq"], s["dk"], s["dv"]
    if op == "paged":
        ra.ra_paged_attn_fwd(s["q"], s["k_pages"], s["v_pages"], s["table"], s["seq_lens"], s["cu"], s["o"], s["lse"],
                             max_new=s["new_max"], max_len=s["len_max"], window=s["W"], sinks=s["sinks"],
                             workspace=s["ws"])
        return s["o"], s["lse"]
    ra.ra_paged_append(s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["table"], s["seq_lens"], s["cu"],
                       workspace=s["ws"])
    return s["k_pages"], s["v_pages"]


# ------------------------------------------------------------------ what a pass cannot do without
def _row_pairs(p, W, sinks):
    """How many keys a query at position p of its sequence sees."""
    if not W or W > p:
        return p + 1
    return W + min(sinks, p + 1 - W)


def _sum_pairs(a, b, W, sinks):
    """The sum of _row_pairs over positions a .. b - 1."""
    def upto(x):       # positions 0 .. x - 1
        if not W or x <= W:
            return x * (x + 1) // 2
        rest = x - W   # positions W .. x - 1 see W + min(sinks, 1 .. rest)
        k = min(rest, sinks)
        return W * (W + 1) // 2 + rest * W + k * (k + 1) // 2 + (rest - k) * sinks
    return upto(b) - upto(a)


def work(case):
    if case["op"] in ("window_fwd", "window_bwd"):
        pairs = case["H"] * sum(_sum_pairs(0, n, case["W"], case["sinks"]) for n in _lens(case))
        rows = case["B"] * case["L"]
        qo, kv, lse = rows * case["H"] * case["d"] * 2, rows * case["Hkv"] * case["d"] * 2, rows * case["H"] * 4
        if case["op"] == "window_fwd":
            return {"bytes": 2 * qo + 2 * kv + lse, "flops": 4 * case["d"] * pairs}
        return {"bytes": 4 * qo + 4 * kv + lse, "flops": 10 * case["d"] * pairs}
    new, total = _lens(case)
    token = case["Hkv"] * case["d"] * 2
    if case["op"] == "append":
        return {"bytes": 4 * sum(new) * token, "flops": 0}
    W, sinks = case["W"], case["sinks"]
    read = sum(t if not W else min(t, (k - 1) + min(W, t - k + 1) + min(sinks, max(0, t - k + 1 - W)))
               for k, t in zip(new, total))
    pairs = case["H"] * sum(_sum_pairs(t - k, t, W, sinks) for k, t in zip(new, total))
    rows = sum(new) * case["H"]
    return {"bytes": 2 * read * token + rows * (4 * case["d"] + 4), "flops": 4 * case["d"] * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
def _attend64(q, k, v, pos, W, sinks):
    """q [H, r, d] at positions pos [r], over k, v [Hkv, t, d] of positions 0 .. t - 1 of the same sequence."""
    H, Hkv = q.shape[0], k.shape[0]
    last = int(pos[-1])
    lo = max(0, int(pos[0]) - W + 1) if W else 0
    at = torch.arange(lo, last + 1, device=q.device)
    if sinks and lo > 0:
        at = torch.cat([torch.arange(min(sinks, lo), device=q.device), at])
    ke, ve = k[:, at].double(), v[:, at].double()
    ok = at[None, :] <= pos[:, None]
    if W:
        ok &= (at[None, :] > pos[:, None] - W) | (at[None, :] < sinks)
    qg = q.double().reshape(Hkv, -1, q.shape[2])                                        # [Hkv, G * r, d]
    x = torch.einsum("hrd,htd->hrt", qg, ke) / math.sqrt(q.shape[2])
    x = x.reshape(H, q.shape[1], -1)
    x[:, ~ok] = _NEG
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[..., None])
    o = torch.einsum("hrt,htd->hrd", p.reshape(Hkv, -1, p.shape[2]), ve).reshape(q.shape)
    return at, p, o, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("window_fwd", "window_bwd"):
        H, Hkv, W, sinks, scale = case["H"], case["Hkv"], case["W"], case["sinks"], case["d"] ** -0.5
        grads = case["op"] == "window_bwd"
        if case["B"] * H * case["L"] * min(case["L"], W + 512) * case["d"] * (16 if grads else 6) > 1e13:
            return None
        runs = [(b, 0, case["L"]) for b in range(case["B"])]
        if s["cu"] is not None:
            e = s["cu"].tolist()
            runs = [(0, x, y) for x, y in zip(e, e[1:])]
        if grads:
            dq, dk, dv = (torch.zeros(s[x].shape, dtype=torch.float64, device="cuda") for x in ("q", "k", "v"))
        else:
            o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
            lse = torch.empty((case["B"], H, case["L"]), dtype=torch.float64, device="cuda")
        for b, x, y in runs:
            k, v = (s[t][b, x:y].permute(1, 0, 2) for t in ("k", "v"))
            for r0 in range(0, y - x, 512):
                r1 = min(y - x, r0 + 512)
                q = s["q"][b, x + r0: x + r1].permute(1, 0, 2)
                at, p, oo, ll = _attend64(q, k, v, torch.arange(r0, r1, device="cuda"), W, sinks)
                if not grads:
                    o[b, x + r0: x + r1], lse[b, :, x + r0: x + r1] = oo.permute(1, 0, 2), ll
                    continue
                do = s["do"][b, x + r0: x + r1].permute(1, 0, 2).double()
                pg, dog, qg = (t.reshape(Hkv, -1, t.shape[2]) for t in (p, do, q.double()))
                dp = torch.einsum("hrd,htd->hrt", dog, v[:, at].double())
                ds = pg * (dp - (do * oo).sum(-1).reshape(Hkv, -1, 1)) * scale
                dq[b, x + r0: x + r1] = torch.einsum("hrt,htd->hrd", ds, k[:, at].double()).reshape(do.shape).permute(1, 0, 2)
                dk[b, x + at] += torch.einsum("hrt,hrd->htd", ds, qg).permute(1, 0, 2)
                dv[b, x + at] += torch.einsum("hrt,hrd->htd", pg, dog).permute(1, 0, 2)
        return (dq, dk, dv) if grads else (o, lse)
    if case["op"] == "append":
        k, v = s["k_pages"].double(), s["v_pages"].double()
        t = 0
        for i, (new, total) in enumerate(zip(s["new"], s["total"])):
            for j in range(total - new, total):
                page = int(s["table"][i, j // case["page"]]) if j % case["page"] == 0 or j == total - new else page
                k[page, j % case["page"]], v[page, j % case["page"]] = s["k_new"][t].double(), s["v_new"][t].double()
                t += 1
        return k, v
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty((case["H"], s["T"]), dtype=torch.float64, device="cuda")
    t = 0
    for i, (new, total) in enumerate(zip(s["new"], s["total"])):
        pages = s["table"][i, : -(-total // case["page"])].long()
        k, v = (x[pages].reshape(-1, case["Hkv"], case["d"])[:total].permute(1, 0, 2) for x in (s["k_pages"], s["v_pages"]))
        for r0 in range(0, new, 64):
            r1 = min(new, r0 + 64)
            q = s["q"][t + r0: t + r1].permute(1, 0, 2)
            pos = torch.arange(total - new + r0, total - new + r1, device="cuda")
            _, _, oo, ll = _attend64(q, k, v, pos, case["W"], case["sinks"])
            o[t + r0: t + r1], lse[:, t + r0: t + r1] = oo.permute(1, 0, 2), ll
        t += new
    return o, lse
