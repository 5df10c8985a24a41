"""prefill_paged_varlen where one piece of work takes much longer than a wait
may, and where counts of keys come near 2^31."""

import math

import pytest
import torch

from exact_softmax_attention_causal_b200 import prefill_paged_varlen

pytestmark = pytest.mark.gpu

BF16, I32 = torch.bfloat16, torch.int32


def test_a_piece_may_take_longer_than_a_wait(monkeypatch):
    """A wait's budget is for one step of the pipeline, not for a whole item. Every multiprocessor's share is one item
    of 300 key tiles (at least 300 x 2,000 cycles: four products of 128 x 128 x 64 and 128 exponentials a row), then
    eight short ones; the budget is 200,000 cycles, 100 us, more than any single step takes."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    Hq, Hkv, d, bs, long_n, long_c, short_c = 4, 1, 64, 128, 64, 300 * 128, 16
    g = torch.Generator("cuda").manual_seed(3)
    blocks = long_c // bs
    kc, vc = (torch.randn((blocks, bs, Hkv, d), generator=g, device="cuda").to(BF16) for _ in range(2))
    table = torch.arange(blocks, dtype=I32, device="cuda").repeat(9 * sms, 1)  # all sequences share the blocks
    n = torch.tensor([long_n] + [1] * 8).repeat(sms)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).to(I32).cuda()
    lens = torch.tensor([long_c] + [short_c] * 8, dtype=I32).repeat(sms).cuda()
    unit = torch.randn((long_n + 8, Hq, d), generator=g, device="cuda").to(BF16)
    status = torch.zeros(1, dtype=I32, device="cuda")
    args = unit.repeat(sms, 1, 1), kc, vc, table, cu, lens, long_c
    prefill_paged_varlen(*args)  # the first launch, without a limit
    monkeypatch.setenv("ATTN_WAIT_BUDGET_CYCLES", "200000")
    o, lse = prefill_paged_varlen(*args, status=status)
    torch.cuda.synchronize()
    monkeypatch.delenv("ATTN_WAIT_BUDGET_CYCLES")
    assert int(status.item()) == 0
    # tolerances as in the tests of the ragged attention: bf16 probabilities and outputs
    k, v = kc.view(-1, d).double(), vc.view(-1, d).double()
    q = unit.double()
    o, lse = o.view(sms, long_n + 8, Hq, d), lse.view(sms, long_n + 8, Hq)
    for rows, c, last in ((slice(0, long_n), long_c, True), (slice(long_n, None), short_c, False)):
        s = torch.einsum("nhd,cd->nhc", q[rows], k[:c]) / math.sqrt(d)
        big = torch.einsum("nhd,cd->nhc", q[rows].abs(), k[:c].abs()).amax(-1) / math.sqrt(d)
        if last:
            i, j = torch.arange(c - long_n, c, device="cuda")[:, None], torch.arange(c, device="cuda")[None]
            s = s.masked_fill((j > i)[:, None], -math.inf)
        rl = torch.logsumexp(s, -1)
        p = (s - rl[..., None]).exp()
        ro, spread = p @ v[:c], p @ v[:c].abs()
        so = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -15 + 2.0 ** -17 * big[..., None]) * spread
        # 38,400 terms in fp32: up to 2^-24 of the sum each for a sum that grows term by term
        sl = 2.0 ** -18 * (big + 1 + rl.abs()) + c * 2.0 ** -24
        assert ((o[:, rows].double() - ro).abs() <= so + c * 2.0 ** -24 * spread).all()
        assert ((lse[:, rows].double() - rl).abs() <= sl).all()


@pytest.mark.parametrize("window,n_sink,hidden", [(2 ** 30 - 1, 2 ** 30, 0), (2 ** 30 - 1, 2 ** 31 - 1, 0), (1, 2 ** 30 - 1, 0),
                                                  (2 ** 29, 2 ** 29, 0), (2 ** 29, 2 ** 29 - 128, 128)])
def test_window_and_sinks_of_the_longest_sequence(window, n_sink, hidden):
    """The newest of 2^30 positions, every block the same, scores of 0: the output is the mean of V, the logarithm of
    the sum that of the number of visible keys. Counts are whole numbers, exact in fp32 up to 2^24 of a multiprocessor's
    stretch; the join adds under 200 of them, 2^-24 of the sum each."""
    bs, d, c = 128, 64, 2 ** 30
    kc = torch.zeros((2, bs, 1, d), dtype=BF16, device="cuda")
    vc = torch.zeros_like(kc)
    t, e = torch.arange(bs, device="cuda")[:, None], torch.arange(d, device="cuda")[None]
    vc[1, :, 0] = ((t * (e + 1)) % 7 < 3).to(BF16)
    table = torch.ones((2, c // bs), dtype=I32, device="cuda")
    if hidden:  # the one block that the newest position does not see
        table[0, (c - window - hidden) // bs] = -1
    cu, lens = torch.tensor([0, 1, 6], dtype=I32, device="cuda"), torch.tensor([c, 40], dtype=I32, device="cuda")
    q = torch.ones((6, 2, d), dtype=BF16, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    o, lse = prefill_paged_varlen(q, kc, vc, table, cu, lens, c, mask="window", window=window, n_sink=n_sink, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    mean = vc[1, :, 0].double().mean(0)
    slack = 200 * 2.0 ** -24
    assert ((o[0].double() - mean).abs() <= (2.0 ** -8 + slack) * mean).all()
    assert ((lse[0].double() - math.log(c - hidden)).abs() <= slack + 2.0 ** -18 * 22).all()
    for i in range(5):  # the short sequence beside it: positions 35 to 39
        seen = torch.arange(36 + i, device="cuda")
        seen = seen[(35 + i - seen < window) | (seen < n_sink)]
        mean = vc[1, seen, 0].double().mean(0)
        assert ((o[1 + i].double() - mean).abs() <= (2.0 ** -8 + slack) * mean).all()
        assert ((lse[1 + i].double() - math.log(len(seen))).abs() <= slack + 2.0 ** -18 * 5).all()
