"""The bound that include/ra.h gives for ra_window_attn_bwd_workspace_bytes."""
import itertools

import pytest

SIZES = list(itertools.product((1, 4), (1, 127, 5000, 8192, 131072), (1, 8, 32), (64, 128), (1, 1024), (0, 4, 64, 512, 4096),
                               (0, 1, 30, 500)))


def bound(B, L, H, H_kv, d, sinks, n_seqs):
    """The status word, D (both in whole 256 bytes), and the sinks' partial gradients: 32 MiB, or two parts
    of each sequence and two more, one at least of them a chunk's."""
    slots = (2 * n_seqs + 3) * 8 * B * H_kv * min(sinks, L) * d
    return 256 + -(-4 * B * L * H // 256) * 256 + -(-max(32 << 20, slots) // 256) * 256


@pytest.mark.parametrize("heads", [1, 4])
def test_workspace_stays_inside_its_bound(ralib, heads):
    for B, L, H_kv, d, window, sinks, n_seqs in SIZES:
        if B > 1 and n_seqs:
            continue
        need = ralib.ra_window_attn_bwd_workspace_bytes(B, L, heads * H_kv, H_kv, d, window, sinks, n_seqs)
        assert 0 < need <= bound(B, L, heads * H_kv, H_kv, d, sinks, n_seqs), (B, L, H_kv, d, window, sinks, n_seqs)


def test_what_passes_32_mib(ralib):
    """Many sinks and heads do without packing, and so do many sequences."""
    f = ralib.ra_window_attn_bwd_workspace_bytes
    plain = lambda B, L, H: 256 + 4 * B * L * H
    assert f(1, 131072, 8, 8, 128, 1024, 4096) - plain(1, 131072, 8) == 96 << 20
    assert f(4, 8192, 32, 32, 128, 100, 512) - plain(4, 8192, 32) == 192 << 20
    # a slot of 512 KiB: two for each of 31 sequences and two more are 32 MiB, with no room for a second chunk
    assert f(1, 100000, 8, 8, 128, 128, 64, 31) - plain(1, 100000, 8) == 32 << 20
    assert f(1, 100000, 8, 8, 128, 128, 64, 32) - plain(1, 100000, 8) == 33 << 20
