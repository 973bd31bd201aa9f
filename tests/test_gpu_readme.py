"""The README's windowed and paged snippets, as they stand there, one after the other."""
import os
import re

import pytest
import torch

from conftest import ROOT
from synthetic_inputs import randn_bf16
from test_gpu_paged import Cache, assert_paged, cu_of

pytestmark = pytest.mark.gpu


def snippet(call):
    """The README's block of Python that makes the call."""
    text = open(os.path.join(ROOT, "README.md")).read()
    found = [b for b in re.findall(r"```python\n(.*?)```", text, flags=re.S) if "ra." + call + "(" in b]
    assert len(found) == 1
    return found[0]


@pytest.mark.parametrize("new,grown", [([1] * 64, 1100), ([300, 1, 17], 9000)], ids=["decode", "chunks"])
def test_a_server_follows_the_readme(ralib, gpu, new, grown):
    B, L, H, H_kv, d, page, n = 1, 2000, 8, 4, 128, 16, len(new)
    q, k, v, do = (randn_bf16((B, L, h, d), h).cuda() for h in (H, H_kv, H_kv, H))
    names = dict(ra=ralib, torch=torch, B=B, L=L, H=H, H_kv=H_kv, d=d, q=q, k=k, v=v, do=do, o=torch.empty_like(q),
                 lse=torch.empty((B, H, L), device="cuda"), dq=torch.empty_like(q), dk=torch.empty_like(k),
                 dv=torch.empty_like(v))
    exec(snippet("ra_window_attn_bwd"), names)
    ralib.ra_check_status(names["ws"])
    # then a batch of new tokens, of this many sequences with this many keys
    lens = [max(x, grown - 13 * s) for s, x in enumerate(new)]
    c = Cache(lens, page, H_kv, d, grown)
    for s, (x, length) in enumerate(zip(new, lens)):
        c.fill(s, 0, length - x)
    T = sum(new)
    names.update(T=T, n=n, k_pages=c.k, v_pages=c.v, block_table=c.table, seq_lens=c.seq_lens, cu=cu_of(new),
                 q=randn_bf16((T, H, d), 5).cuda(), max_new=max(new), max_len=grown,
                 k_new=torch.cat([c.ks[s][m - x:] for s, (x, m) in enumerate(zip(new, lens))]),
                 v_new=torch.cat([c.vs[s][m - x:] for s, (x, m) in enumerate(zip(new, lens))]),
                 o=torch.empty((T, H, d), dtype=torch.bfloat16, device="cuda"), lse=torch.empty((H, T), device="cuda"))
    exec(snippet("ra_paged_append"), names)
    ralib.ra_check_status(names["ws"])
    assert_paged(c, names["q"], names["o"], names["lse"], new, 0, 0)
