"""A NaN among the keys that rows see reaches their O however a call is cut: whole units, pieces joined by
the second kernel, parts of long units, both forms.  (Finite inputs are asked for; a row must not come out
finite without what it should have seen.)"""
import pytest
import torch

from synthetic_inputs import randn_bf16
from test_gpu_paged import Cache, cu_of
from test_gpu_paged_tree import attend, trees_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,H,Hkv,d,length", [
    (40, 8, 2, 128, 100), (40, 8, 2, 128, 9000), (40, 8, 2, 64, 9000), (100, 8, 2, 64, 40000), (100, 8, 2, 128, 40000),
    (8, 8, 2, 128, 700), (8, 8, 2, 64, 9000), (3, 4, 4, 128, 20000)])
@pytest.mark.parametrize("wide", [False, True])
def test_nan_key(ralib, gpu, n, H, Hkv, d, length, wide):
    for at in (5, length // 2, length - n - 1):
        c = Cache([length], 32, Hkv, d, 3)
        c.ks[0][at, Hkv - 1, 7] = float("nan")
        c.fill_all()
        if wide:            # a table for more tokens than are summed in one part
            c.table = torch.nn.functional.pad(c.table, (0, 5000), value=-1).contiguous()
        q = randn_bf16((n, H, d), 4).cuda()
        trees = trees_of([n], "levels")
        o, _, _ = attend(ralib, c, q, cu_of([n]), trees, torch.float32)
        group = H // Hkv
        assert bool(torch.isnan(o[:, H - group:]).all()), at
        assert Hkv == 1 or bool(torch.isfinite(o[:, :H - group]).all()), at
