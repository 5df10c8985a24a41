"""Block-table entries outside the pool in prefill_paged_varlen: NaN in the rows
that see a key of such a block, and in no other row, whatever rows share a tile
with them; the device-check bit in either case."""

import pytest
import torch

from exact_softmax_attention_causal_b200 import prefill_paged_varlen
from test_gpu_prefill_varlen import Batch

pytestmark = pytest.mark.gpu

I32 = torch.int32


def _sees(n, c, bs, block, mask, window, n_sink):
    """Which of the newest n of c positions see a key of the block."""
    i, j = torch.arange(c - n, c)[:, None], torch.arange(block * bs, min(c, (block + 1) * bs))[None]
    seen = torch.ones((n, j.shape[1]), dtype=torch.bool) if mask == "full" else j <= i
    if mask == "window":
        seen = seen & ((i - j < window) | (j < n_sink))
    return seen.any(1)


def _check(b, changes, mask="causal", window=0, n_sink=0):
    """changes: (sequence, block, entry)."""
    args = b.args()
    for s, block, entry in changes:
        args[3][s, block] = entry
    status = torch.zeros(1, dtype=I32, device="cuda")
    o, lse = prefill_paged_varlen(*args, b.max_len, mask=mask, window=window, n_sink=n_sink,
                                  sinks=None if b.sinks is None else b.sinks.cuda(), status=status)
    o, lse = o.cpu(), lse.cpu()
    hit_any = False
    for s, (n, c) in enumerate(zip(b.n, b.ctx)):
        hit = torch.zeros(n, dtype=torch.bool)
        for at, block, _ in changes:
            if at == s:
                hit |= _sees(n, c, b.bs, block, mask, window, n_sink)
        hit_any |= bool(hit.any())
        r = slice(int(b.cu[s]), int(b.cu[s + 1]))
        ro, rl, so, sl = b.ref(s, mask=mask, window=window, n_sink=n_sink)
        assert torch.isnan(o[r][hit].float()).all() and torch.isnan(lse[r][hit]).all(), s
        assert ((o[r].double() - ro).abs() <= so)[~hit].all(), (s, int(torch.isnan(o[r][~hit].float()).sum()))
        assert ((lse[r].double() - rl).abs() <= sl)[~hit].all(), s
    assert int(status.item()) == int(hit_any)


@pytest.mark.parametrize("Hq,Hkv,d,bs", [(8, 2, 128, 16), (4, 1, 64, 32), (8, 8, 64, 128), (6, 2, 128, 64)])
def test_the_newest_block_of_a_chunk(Hq, Hkv, d, bs):
    # the older rows of the same tile do not see it
    b = Batch([300, 7, 40], [300, 90, 40], Hq, Hkv, d, bs, 31, sinks=d == 64)
    _check(b, [(0, 299 // bs, -1), (2, 39 // bs, 10 ** 6)])


def test_a_block_in_the_middle_of_a_chunk():
    b = Batch([300, 5], [700, 600], 8, 2, 128, 16, 32)
    _check(b, [(0, 30, 2 ** 31 - 1), (0, 35, -2 ** 31)])


@pytest.mark.parametrize("n_sink", [0, 5, 200])
def test_blocks_at_both_ends_of_a_window(n_sink):
    # the oldest rows see one, the newest rows the other, those between neither
    b = Batch([200, 9], [900, 500], 8, 2, 64, 16, 33, sinks=True)
    _check(b, [(0, 39, -1), (0, 55, 10 ** 6), (1, 30, 10 ** 6)], mask="window", window=70, n_sink=n_sink)


def test_a_block_of_sink_positions_and_one_that_no_row_sees():
    b = Batch([60, 3], [900, 500], 8, 2, 64, 16, 34)
    _check(b, [(0, 1, -1)], mask="window", window=50, n_sink=20)
    _check(b, [(0, 2, -1), (1, 5, 10 ** 6)], mask="window", window=50, n_sink=20)


def test_an_item_cut_between_multiprocessors():
    b = Batch([64], [6000], 4, 1, 64, 16, 35)
    _check(b, [(0, 5998 // 16, -1)])
    _check(b, [(0, 5945 // 16, -1)])
    b = Batch([6], [9000], 4, 1, 128, 16, 36, sinks=True)  # one tile of rows, its key tiles by two teams
    _check(b, [(0, 8999 // 16, -1)])
    _check(b, [(0, 17, -1)], mask="full")


def test_without_a_mask_every_row_sees_every_block():
    b = Batch([150, 20], [300, 200], 8, 2, 128, 16, 37)
    _check(b, [(0, 18, -1)], mask="full")
