"""Single tokens of as many sequences as a call takes: each (sequence, key/value head) pair is
counted, whatever the number, and every row is written."""
import pytest
import torch

import window_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [(1 << 23) + 5, 1 << 24])
def test_millions_of_sequences(ralib, gpu, n):
    """n sequences share the pages of 64 kinds of cache, of 1 to 32 tokens."""
    kinds, page, d = 64, 16, 64
    g = torch.Generator(device="cuda").manual_seed(n)
    lens = torch.randint(1, 2 * page + 1, (kinds,), generator=g, device="cuda", dtype=torch.int32)
    k, v = (torch.randn((2 * kinds, page, 1, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    kind = torch.arange(n, device="cuda", dtype=torch.int32) % kinds
    table = torch.stack([2 * kind, 2 * kind + 1], 1).contiguous()
    seq_lens = lens[kind.long()].contiguous()
    cu = torch.arange(n + 1, device="cuda", dtype=torch.int32)
    q = torch.empty((n, 1, d), dtype=torch.bfloat16, device="cuda")
    for i in range(0, n, 1 << 20):
        q[i:i + (1 << 20)] = torch.randn(q[i:i + (1 << 20)].shape, generator=g, device="cuda").bfloat16()
    o = torch.full_like(q, float("nan"))
    lse = torch.full((1, n), float("nan"), device="cuda")
    max_len = 20000         # longer than any: runs of the sequences' keys, not a block for each
    ws = ralib.new_workspace(ralib.ra_paged_attn_workspace_bytes(n, n, 1, 1, d, 1, max_len))
    ralib.ra_paged_attn_fwd(q, k, v, table, seq_lens, cu, o, lse, 1, max_len, workspace=ws)
    ralib.ra_check_status(ws)
    assert not bool(torch.isnan(lse).any())
    kd, vd = k.double().reshape(kinds, 2 * page, d), v.double().reshape(kinds, 2 * page, d)
    ok = torch.arange(2 * page, device="cuda")[None, :] < lens[:, None]
    step = kinds << 13
    for i in range(0, n, step):
        rows = q[i:i + step, 0].double()
        m = rows.shape[0]
        pad = torch.zeros((-m % kinds, d), dtype=torch.float64, device="cuda")
        x = torch.cat([rows, pad]).reshape(-1, kinds, d)
        s = (torch.einsum("ncd,ctd->nct", x, kd) * d ** -0.5).masked_fill(~ok, float("-inf"))
        le = torch.logsumexp(s, -1)
        p = torch.exp(s - le[..., None])
        want = torch.einsum("nct,ctd->ncd", p, vd).reshape(-1, d)[:m]
        # P in two bf16 parts: the result's rounding, and EPS for every weight
        tol = ref.U * 1.01 * want.abs() + 2 * ref.EPS * (torch.einsum("nct,ctd->ncd", p, vd.abs()).reshape(-1, d)[:m] + want.abs())
        ref.assert_within(o[i:i + m, 0], want, tol + 1e-6, "O from row %d" % i)
        ref.assert_within(lse[0, i:i + m], le.reshape(-1)[:m], torch.full((m,), ref.EPS, device="cuda", dtype=torch.float64), "LSE")
