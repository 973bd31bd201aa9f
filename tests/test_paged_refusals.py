"""Sizes whose products leave 64 bits are refused by the paged calls, not taken for small ones."""
import pytest

FAKE = 0x10000      # 16-byte aligned, never dereferenced: every call below fails its checks first


def _fwd(lib, **kw):
    a = dict(T=64, n=4, H=8, Hkv=2, d=128, n_pages=10, page=16, pstride=16 * 2 * 128, max_pages=20, qs=1024, new=16, len=300)
    a.update(kw)
    return lib.ra_paged_attn_fwd(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, a["T"], a["n"], a["H"], a["Hkv"], a["d"],
                                 a["n_pages"], a["page"], a["pstride"], a["max_pages"], a["qs"], a["new"], a["len"], 0, 0,
                                 0.0, 0, FAKE, 1 << 40, None)


def _append(lib, **kw):
    a = dict(T=8, n=2, Hkv=2, d=128, n_pages=10, page=16, pstride=4096, max_pages=4, stride=256)
    a.update(kw)
    return lib.ra_paged_append(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, a["T"], a["n"], a["Hkv"], a["d"], a["n_pages"],
                               a["page"], a["pstride"], a["max_pages"], a["stride"], FAKE, 256, None)


BOTH = [dict(max_pages=1 << 60), dict(max_pages=(1 << 60) + 1), dict(max_pages=(1 << 63) - 1), dict(pstride=1 << 62),
        dict(pstride=(1 << 63) - 8), dict(pstride=1 << 39), dict(page=65536, pstride=1 << 25, max_pages=1 << 48)]


@pytest.mark.parametrize("kw", BOTH + [dict(qs=1 << 62), dict(qs=(1 << 63) - 8), dict(qs=1 << 39)])
def test_forward_refuses(ralib, kw):
    assert _fwd(ralib.lib(), **kw) == 3
    assert "beyond the supported range" in ralib.lib().ra_last_error().decode()


@pytest.mark.parametrize("kw", BOTH + [dict(stride=1 << 62), dict(stride=(1 << 63) - 8), dict(stride=1 << 39)])
def test_append_refuses(ralib, kw):
    assert _append(ralib.lib(), **kw) == 3
    assert "beyond the supported range" in ralib.lib().ra_last_error().decode()
