"""Numbers of packed sequences that the windowed kernels' 32-bit unit numbers would not hold are refused."""
import pytest

FAKE = 0x10000      # 16-byte aligned, never dereferenced: every call below fails its checks first


@pytest.mark.parametrize("n", [(1 << 29) + 1, 1 << 30, (1 << 31) - 1])
def test_too_many_sequences(ralib, n):
    lib = ralib.lib()
    sizes = (FAKE, n, 1, 1024, 4, 2, 128, 100)
    assert lib.ra_window_attn_fwd(FAKE, FAKE, FAKE, FAKE, FAKE, *sizes, 0, 0.0, 0, FAKE, 256, None) == 3
    assert "n_seqs" in lib.ra_last_error().decode()
    for sinks in (0, 4):
        assert lib.ra_window_attn_bwd(*[FAKE] * 9, *sizes, sinks, 0.0, 0, FAKE, 1 << 50, None) == 3
        assert "n_seqs" in lib.ra_last_error().decode()
        assert ralib.ra_window_attn_bwd_workspace_bytes(1, 1024, 4, 2, 128, 100, sinks, n) == 0


def test_the_most_sequences(ralib):
    assert ralib.ra_window_attn_bwd_workspace_bytes(1, 1024, 4, 2, 128, 100, 0, 1 << 29) == 256 + 1024 * 4 * 4
