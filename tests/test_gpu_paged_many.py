"""Single tokens of as many sequences as a call takes: each (sequence, key/value head) pair is
counted, whatever the number, every row is written, and the time grows with the sequences."""
import pytest
import torch

import window_reference as ref

pytestmark = pytest.mark.gpu

KINDS, PAGE, D = 64, 16, 64


class Batch:
    """n sequences that share the pages of 64 kinds of cache, of 1 to 32 tokens; one new token each."""

    def __init__(self, n):
        g = torch.Generator(device="cuda").manual_seed(n)
        self.n = n
        self.lens = torch.randint(1, 2 * PAGE + 1, (KINDS,), generator=g, device="cuda", dtype=torch.int32)
        self.k, self.v = (torch.randn((2 * KINDS, PAGE, 1, D), generator=g, device="cuda").bfloat16() for _ in range(2))
        kind = torch.arange(n, device="cuda", dtype=torch.int32) % KINDS
        self.table = torch.stack([2 * kind, 2 * kind + 1], 1).contiguous()
        self.seq_lens = self.lens[kind.long()].contiguous()
        self.cu = torch.arange(n + 1, device="cuda", dtype=torch.int32)
        self.q = torch.empty((n, 1, D), dtype=torch.bfloat16, device="cuda")
        for i in range(0, n, 1 << 20):
            self.q[i:i + (1 << 20)] = torch.randn(self.q[i:i + (1 << 20)].shape, generator=g, device="cuda").bfloat16()
        self.o = torch.full_like(self.q, float("nan"))
        self.lse = torch.full((1, n), float("nan"), device="cuda")

    def attend(self, ra, max_len):
        ws = ra.new_workspace(ra.ra_paged_attn_workspace_bytes(self.n, self.n, 1, 1, D, 1, max_len))

        def call():
            ra.ra_paged_attn_fwd(self.q, self.k, self.v, self.table, self.seq_lens, self.cu, self.o, self.lse, 1, max_len,
                                 workspace=ws)

        call()
        ra.ra_check_status(ws)
        return call

    def check(self):
        assert not bool(torch.isnan(self.lse).any())
        kd, vd = (x.double().reshape(KINDS, 2 * PAGE, D) for x in (self.k, self.v))
        ok = torch.arange(2 * PAGE, device="cuda")[None, :] < self.lens[:, None]
        step = KINDS << 13
        for i in range(0, self.n, step):
            rows = self.q[i:i + step, 0].double()
            m = rows.shape[0]
            pad = torch.zeros((-m % KINDS, D), dtype=torch.float64, device="cuda")
            x = torch.cat([rows, pad]).reshape(-1, KINDS, D)
            s = (torch.einsum("ncd,ctd->nct", x, kd) * D ** -0.5).masked_fill(~ok, float("-inf"))
            le = torch.logsumexp(s, -1)
            p = torch.exp(s - le[..., None])
            flat = lambda y: torch.einsum("nct,ctd->ncd", p, y).reshape(-1, D)[:m]
            want = flat(vd)
            # P in two bf16 parts: the result's rounding, and EPS for every weight
            tol = ref.U * 1.01 * want.abs() + 2 * ref.EPS * (flat(vd.abs()) + want.abs()) + 1e-6
            ref.assert_within(self.o[i:i + m, 0], want, tol, "O from row %d" % i)
            le = le.reshape(-1)[:m]
            ref.assert_within(self.lse[0, i:i + m], le, torch.full_like(le, ref.EPS), "LSE from row %d" % i)


@pytest.mark.parametrize("n", [(1 << 23) + 5, 1 << 24])
def test_millions_of_sequences(ralib, gpu, n):
    b = Batch(n)
    b.attend(ralib, 20000)         # longer than any: runs of the sequences' keys, not a block for each
    b.check()


def test_time_grows_with_the_sequences(ralib, gpu):
    """Eight times as many short sequences take about eight times as long (and not 64 times, as where
    each sequence's block looks at all of them)."""
    times = []
    for n in (1 << 14, 1 << 17):
        b = Batch(n)
        call = b.attend(ralib, 32)
        b.check()
        best = float("inf")
        for _ in range(5):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            call()
            end.record()
            torch.cuda.synchronize()
            best = min(best, start.elapsed_time(end))
        times.append(best)
    assert times[1] < 20 * times[0], times


@pytest.mark.parametrize("n,longest", [(512, 300), (513, 300), (700, 40), (2000, 1000)])
def test_short_sequences(ralib, gpu, n, longest):
    """A block for each pair, or runs of all of them: the same rows."""
    b = Batch(n)
    b.attend(ralib, longest)
    b.check()
