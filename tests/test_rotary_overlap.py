"""ra_paged_append_rotary refuses rotated queries that would overlap what the call still reads, and takes
the columns of one fused projection.  (On the CPU: the workspace of each call is too small, which is found
last.)"""
import random

import pytest

BASE = 1 << 20      # 16-byte aligned, never dereferenced


def call(lib, q, k, v, out, T, H, Hkv, d, qs, outs, stride):
    """Addresses in elements of 2 bytes; 'workspace' or 'overlap'."""
    far = BASE << 8
    status = lib.ra_paged_append_rotary(BASE + 2 * q, BASE + 2 * k, BASE + 2 * v, BASE + 2 * out, far, far, far, far, far, 0, far, T, 2,
                                        H, Hkv, d, 16, 10, 16, 16 * Hkv * d, 4, qs, outs, stride, 0, far, 16, None)
    assert status == 1
    message = lib.ra_last_error().decode()
    assert ("workspace" in message) != ("overlap" in message), message
    return "workspace" if "workspace" in message else "overlap"


H, HKV, D, T = 4, 2, 64, 6
ROW = (H + 2 * HKV) * D                     # a token of a fused projection: q, k, v
K, V = H * D, (H + HKV) * D


@pytest.mark.parametrize("out,outs,verdict", [
    (0, ROW, "workspace"),                                  # in place
    (D, ROW, "overlap"), (ROW, ROW, "overlap"),             # q's columns a head on, a token on
    (K, ROW, "overlap"), (V, ROW, "overlap"),               # the keys', the values'
    (K - 3 * D, ROW, "overlap"), (V - 7 * D, ROW, "overlap"),
    (T * ROW, ROW, "workspace"), (T * ROW - D, ROW, "overlap"), (T * ROW, H * D, "workspace"),
    (T * ROW - HKV * D, H * D, "overlap"), (T * ROW - HKV * D + D, H * D, "overlap"),
    (96, H * D, "overlap"), (-T * H * D, H * D, "workspace"), (8 - T * H * D, H * D, "overlap"),
])
def test_fused_projection(ralib, out, outs, verdict):
    assert call(ralib.lib(), 0, K, V, out, T, H, HKV, D, ROW, outs, ROW) == verdict


def test_columns_beside_them(ralib):
    """A projection with room for the rotated queries in each token's row, before, between or behind."""
    wide = ROW + H * D
    for q, k, v, out in ((0, K, V, ROW), (H * D, H * D + K, H * D + V, 0), (0, 2 * K, 2 * K + HKV * D, K)):
        assert call(ralib.lib(), q, k, v, out, T, H, HKV, D, wide, wide, wide) == "workspace"
        assert call(ralib.lib(), q, k, v, out, T, H, HKV, D, wide, wide + 8, wide) == "overlap"
        assert call(ralib.lib(), q, k, v, out, 1, H, HKV, D, wide, 8 * wide, wide) == "workspace"
    # one token: strides do not matter, and in place needs none
    assert call(ralib.lib(), 0, K, V, 0, 1, H, HKV, D, ROW, 2 * ROW, ROW) == "workspace"
    # rows that lie in the gaps of twice as far rows
    assert call(ralib.lib(), 0, 100 * ROW, 200 * ROW, 2 * K, T, H, HKV, D, 4 * K, 2 * K, ROW) == "overlap"
    assert call(ralib.lib(), 0, 100 * ROW, 200 * ROW, K, T, H, HKV, D, 4 * K, 2 * K, ROW) == "workspace"
    assert call(ralib.lib(), 0, 100 * ROW, 200 * ROW, K, T, H, HKV, D, 2 * K, 4 * K, ROW) == "workspace"


def test_the_largest_strides(ralib):
    big = (1 << 39) - 8
    assert call(ralib.lib(), 0, K, V, 0, 1 << 24, H, HKV, D, big, big, big) == "workspace"
    assert call(ralib.lib(), 0, K, V, D, 1 << 24, H, HKV, D, big, big, big) == "overlap"
    assert call(ralib.lib(), 0, K, V, V + HKV * D, 1 << 24, H, HKV, D, big, big, big) == "workspace"


def test_against_all_elements(ralib):
    """Random strides and places against the sets of all elements."""
    r = random.Random(5)
    verdicts = set()
    for _ in range(3000):
        n, h, kv = r.randint(1, 5), r.choice([1, 2, 3]), r.choice([1, 2])
        qs, outs, ks = (r.choice([64 * x + 8 * r.randint(0, 3) for x in (a, a + 1, 2 * a, 3 * a + 2)]) for a in (h, h, kv))
        if r.random() < 0.5:
            outs = qs
        q, k, v, out = (8 * r.randint(0, 120) for _ in range(4))
        rows = lambda at, stride, width: {at + i * stride + x for i in range(n) for x in range(0, width, 8)}    # noqa: E731
        o = rows(out, outs, h * 64)
        same = q == out and (qs == outs or n == 1)
        if q == out and not same:
            continue
        meets = bool(o & rows(k, ks, kv * 64) or o & rows(v, ks, kv * 64) or (o & rows(q, qs, h * 64) and not same))
        got = call(ralib.lib(), q, k, v, out, n, h, kv, 64, qs, outs, ks)
        assert got == ("overlap" if meets else "workspace"), (n, h, kv, qs, outs, ks, q, k, v, out)
        verdicts.add(got)
    assert len(verdicts) == 2
