"""prefill_paged_varlen against softmax attention in 64 bits, sequence by
sequence, at the lengths, head groups and masks where it can go wrong.

Tolerances. A probability is rounded to bf16 once, 2^-8 of itself, so the
output is off by 2^-8 of sum p |v| / l at most, and by 2^-8 of itself from its
own rounding. What fp32 leaves is far below: with A the largest
scale * sum |q_i k_i| of a row, a score is off by less than 2^-18 A (8 steps of
16 products, each step's sum truncated at 2^-22 of its largest term, and 2^-23
of the score from the scaled exponent), its exponential by 2^-21 besides, and
the row's sums over n keys by n 2^-24. So o may be off by
2^-8 |o| + (2^-8 + 2^-15 + 2^-17 A) sum p |v| / l, and lse by 2^-18 (A + 1 + |lse|).
A factor below fp32's smallest normal number, 2^-126, may become 0 (next to a
sink logit of 200 the whole output is of that kind): that takes away at most
2^-126 of the largest |v|, which is below 2^6 here, so 2^-120 is allowed besides.
"""

import math

import pytest
import torch

from exact_softmax_attention_causal_b200 import (AttnError, decode_paged, decode_paged_window, prefill_paged,
                                                  prefill_paged_varlen, prefill_paged_varlen_workspace_bytes)

pytestmark = pytest.mark.gpu

BF16, I32 = torch.bfloat16, torch.int32
NAN = float("nan")


class Batch:
    """Rows and contexts of a batch, its cache in a shuffled pool: NaN wherever no token is."""

    def __init__(self, n, ctx, Hq, Hkv, d, bs, seed=0, sinks=False, scale_q=1.0):
        g = torch.Generator().manual_seed(seed)
        self.n, self.ctx, self.Hq, self.Hkv, self.d, self.bs = n, ctx, Hq, Hkv, d, bs
        self.T, self.max_len = sum(n), max(1, max(ctx))
        self.q = (torch.randn((self.T, Hq, d), generator=g) * scale_q).to(BF16)
        blocks = [-(-c // bs) for c in ctx]
        nb = sum(blocks) + 3
        perm = torch.randperm(nb, generator=g).to(I32)
        self.k_cache = torch.full((nb, bs, Hkv, d), NAN, dtype=BF16)
        self.v_cache = torch.full((nb, bs, Hkv, d), NAN, dtype=BF16)
        self.table = torch.full((len(n), -(-self.max_len // bs) + 1), -1, dtype=I32)
        self.k, self.v, at = [], [], 0
        for b, c in enumerate(ctx):
            self.table[b, :blocks[b]] = perm[at:at + blocks[b]]
            k, v = (torch.randn((c, Hkv, d), generator=g).to(BF16) for _ in range(2))
            t = torch.arange(c)
            where = self.table[b].long()[t // bs], t % bs
            self.k_cache[where], self.v_cache[where] = k, v
            self.k.append(k)
            self.v.append(v)
            at += blocks[b]
        self.cu = torch.tensor([0] + list(torch.tensor(n).cumsum(0)), dtype=I32)
        self.seq_lens = torch.tensor(ctx, dtype=I32)
        self.sinks = torch.rand(Hq, generator=g) * 7 - 1 if sinks else None

    def args(self):
        return [t.cuda() for t in (self.q, self.k_cache, self.v_cache, self.table, self.cu, self.seq_lens)]

    def run(self, mask="causal", window=0, n_sink=0, status=None, **kw):
        return prefill_paged_varlen(*self.args(), self.max_len, mask=mask, window=window, n_sink=n_sink,
                                    sinks=None if self.sinks is None else self.sinks.cuda(), status=status, **kw)

    def ref(self, b, mask="causal", window=0, n_sink=0, scale=None):
        """(o, lse, slack of o, slack of lse) of sequence b's rows."""
        n, c, group = self.n[b], self.ctx[b], self.Hq // self.Hkv
        r0 = int(self.cu[b])
        scale = 1 / math.sqrt(self.d) if scale is None else scale
        q = self.q[r0:r0 + n].double()
        k, v = (t.double().repeat_interleave(group, 1) for t in (self.k[b], self.v[b]))
        s = torch.einsum("nhd,chd->hnc", q, k) * scale
        big = torch.einsum("nhd,chd->hnc", q.abs(), k.abs()).amax(-1).t() * scale
        i, j = torch.arange(c - n, c)[:, None], torch.arange(c)[None]
        seen = torch.ones((n, c), dtype=torch.bool)
        if mask != "full":
            seen &= j <= i
        if mask == "window":
            seen &= (i - j < window) | (j < n_sink)
        s = s.masked_fill(~seen, -math.inf)
        if self.sinks is not None:
            s = torch.cat([s, self.sinks.double()[:, None, None].expand(-1, n, 1)], -1)
        lse = torch.logsumexp(s, -1)
        p = (s - lse[..., None]).exp()[..., :c]
        o = torch.einsum("hnc,chd->nhd", p, v)
        spread = torch.einsum("hnc,chd->nhd", p, v.abs())
        lse = lse.t()
        so = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -15 + 2.0 ** -17 * big[..., None]) * spread + 2.0 ** -120
        return o, lse, so, 2.0 ** -18 * (big + 1 + lse.abs())

    def check(self, o, lse, seqs=None, **kw):
        for b in range(len(self.n)) if seqs is None else seqs:
            if self.n[b] == 0:
                continue
            ro, rl, so, sl = self.ref(b, **kw)
            r = slice(int(self.cu[b]), int(self.cu[b + 1]))
            eo, el = (o[r].double().cpu() - ro).abs(), (lse[r].double().cpu() - rl).abs()
            assert (eo <= so).all(), (b, "o", float((eo - so).max()), int((~(eo <= so)).sum()))
            assert (el <= sl).all(), (b, "lse", float((el - sl).max()))

    def run_and_check(self, **kw):
        status = torch.zeros(1, dtype=I32, device="cuda")
        o, lse = self.run(status=status, **kw)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        self.check(o, lse, **kw)
        return o, lse


MASKS = [dict(mask="causal"), dict(mask="full"), dict(mask="window", window=1), dict(mask="window", window=100),
         dict(mask="window", window=130, n_sink=4), dict(mask="window", window=37, n_sink=300)]


@pytest.mark.parametrize("d", [64, 128])
def test_one_token(d):
    for ctx in (1, 2, 17, 128, 129, 700):
        Batch([1], [ctx], 4, 1, d, 16, ctx).run_and_check()


@pytest.mark.parametrize("kw", MASKS)
@pytest.mark.parametrize("Hq,Hkv,d,bs", [(8, 2, 128, 16), (8, 8, 64, 32), (16, 2, 64, 128), (6, 2, 128, 64)])
def test_mixed_batch(kw, Hq, Hkv, d, bs):
    n = [1, 0, 5, 130, 1, 33, 64, 0, 200, 300]
    ctx = [900, 40, 5, 611, 1, 300, 64, 0, 1000, 301]
    Batch(n, ctx, Hq, Hkv, d, bs, 3, sinks=bs == 128).run_and_check(**kw)


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 16, 48, 100, 128, 150])
@pytest.mark.parametrize("d", [64, 128])
def test_head_groups(group, d):
    # rows of a tile that no (token, head) pair fills, and groups of more than one tile
    Hkv = 2 if group < 16 else 1
    b = Batch([1, 3, 70], [200, 50, 333], group * Hkv, Hkv, d, 16, group, sinks=group % 2 == 1)
    b.run_and_check()
    b.run_and_check(mask="window", window=40, n_sink=2)


@pytest.mark.parametrize("n,ctx,Hq,Hkv,d", [([1], [20000], 8, 1, 128), ([8], [9000], 4, 2, 64), ([40], [7000], 4, 1, 128),
                                            ([300], [6000], 8, 2, 64), ([1, 1, 9], [5000, 12000, 6001], 16, 4, 128)])
@pytest.mark.parametrize("kw", [dict(), dict(mask="full"), dict(mask="window", window=4000, n_sink=200)])
def test_contexts_cut_between_multiprocessors(n, ctx, Hq, Hkv, d, kw):
    Batch(n, ctx, Hq, Hkv, d, 16, 5, sinks=d == 64).run_and_check(**kw)


def test_many_sequences():
    g = torch.Generator().manual_seed(1)
    n = torch.randint(0, 3, (1000,), generator=g).tolist()
    ctx = [max(c, m) for c, m in zip(torch.randint(0, 60, (1000,), generator=g).tolist(), n)]
    Batch(n, ctx, 2, 1, 64, 16, 2).run_and_check()


def test_long_chunks():
    Batch([1500, 3, 700], [1600, 2000, 700], 8, 1, 64, 128, 6).run_and_check()


def test_large_and_small_scores():
    # a softmax that one key wins, and one that is flat
    Batch([5, 90], [700, 800], 4, 2, 128, 16, 7, scale_q=30.0, sinks=True).run_and_check()
    Batch([5, 90], [700, 800], 4, 2, 128, 16, 8, scale_q=0.001).run_and_check()


def test_sink_logits_far_from_the_scores():
    b = Batch([2, 70], [300, 400], 4, 2, 64, 16, 9, sinks=True)
    for values in ([-math.inf] * 4, [-200.0, 200.0, 90.0, -90.0]):
        b.sinks = torch.tensor(values)
        b.run_and_check()


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_sink_logits_that_are_none_are_flagged(value):
    b = Batch([2, 70, 1], [300, 400, 9000], 4, 2, 64, 16, 9, sinks=True)
    b.sinks[1] = value
    status = torch.zeros(1, dtype=I32, device="cuda")
    o, lse = b.run(status=status)
    assert int(status.item()) == 1
    assert torch.isnan(o[:, 1].float()).all() and torch.isnan(lse[:, 1]).all()
    assert torch.isfinite(o[:, [0, 2, 3]].float()).all() and torch.isfinite(lse[:, [0, 2, 3]]).all()


@pytest.mark.parametrize("n_sink", [30, 39, 40, 41, 1000])
def test_more_sink_positions_than_a_sequence_has(n_sink):
    Batch([3, 40, 1, 7], [40, 40, 5, 33], 4, 2, 64, 16, 23).run_and_check(mask="window", window=6, n_sink=n_sink)


def test_blocks_that_no_row_sees_are_not_read():
    """A window's dropped blocks: entries of -1, and blocks full of NaN."""
    b = Batch([3, 100], [1000, 1500], 8, 2, 64, 16, 10)
    for s, (n, c) in enumerate(zip(b.n, b.ctx)):
        lo = (c - n - 200 + 1) // 16  # the first block a window of 200 reaches, from the oldest row
        gone = b.table[s, 1:lo].clone().long()
        b.k_cache[gone] = NAN
        b.v_cache[gone] = NAN
        b.table[s, 1:lo:2] = -1
    b.run_and_check(mask="window", window=200, n_sink=16)


def test_rows_outside_the_batch_stay():
    b = Batch([4, 0, 50], [100, 7, 300], 8, 2, 128, 16, 11)
    o = torch.full((b.T + 40, 8, 128), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((b.T + 40, 8), 7.0, device="cuda")
    q, *rest = b.args()
    rest[3] += 3  # rows before the first sequence too
    qq = torch.full_like(o, NAN)
    qq[3:3 + b.T] = q
    prefill_paged_varlen(qq, *rest, b.max_len, out=o, lse=lse)
    b.check(o[3:3 + b.T], lse[3:3 + b.T])
    for t in (o, lse):
        assert (t[:3] == 7).all() and (t[3 + b.T:] == 7).all()


def test_bad_lengths_offsets_and_entries_are_flagged():
    n, ctx = [4, 1, 50, 2, 3, 6], [100, 7, 300, 900, 20, 500]
    b = Batch(n, ctx, 8, 2, 128, 16, 12)

    def call(change, bad):
        a = b.args()
        change(a)
        status = torch.zeros(1, dtype=I32, device="cuda")
        o, lse = prefill_paged_varlen(*a, b.max_len, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 1
        b.check(o, lse, [s for s in range(6) if s not in bad])
        for s in bad:
            r = slice(int(b.cu[s]), int(b.cu[s + 1]))
            assert torch.isnan(o[r].float()).all() and torch.isnan(lse[r]).all(), s

    call(lambda a: a[5].__setitem__(2, 49), [2])       # fewer cached tokens than rows
    call(lambda a: a[5].__setitem__(0, -101), [0])     # as a failed extension leaves it
    call(lambda a: a[5].__setitem__(3, 901), [3])      # above max_seq_len
    call(lambda a: a[3].__setitem__((5, 3), 10 ** 6), [5])
    call(lambda a: a[3].__setitem__((2, 0), -1), [2])
    # offsets: a negative one, one past T, two out of order (rows of two sequences)
    for at, value in ((1, -5), (3, 10 ** 6), (3, 2)):
        a = b.args()
        a[4][at] = value
        status = torch.zeros(1, dtype=I32, device="cuda")
        prefill_paged_varlen(*a, b.max_len, status=status)
        assert int(status.item()) == 1


def test_all_sequences_empty():
    b = Batch([0, 0], [5, 0], 4, 1, 64, 16, 13)
    q = torch.zeros((6, 4, 64), dtype=BF16, device="cuda")
    out, lse = torch.full_like(q, 3.0), torch.full((6, 4), 3.0, device="cuda")
    prefill_paged_varlen(q, *b.args()[1:], 5, out=out, lse=lse)
    assert (out == 3).all() and (lse == 3).all()
    o, l = prefill_paged_varlen(*b.args(), 5)
    assert o.shape == (0, 4, 64) and l.shape == (0, 4)


def test_same_bits_on_every_run_and_without_lse():
    b = Batch([1, 200, 7, 1], [9000, 4000, 700, 100], 8, 2, 128, 16, 14)
    o, lse = b.run()
    for _ in range(5):
        o2, l2 = b.run()
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    o3, none = b.run(return_lse=False)
    assert none is None and torch.equal(o, o3)


def test_agrees_with_the_other_entry_points():
    b = Batch([1] * 5, [1, 300, 777, 2048, 64], 8, 2, 64, 16, 15, sinks=True)
    q, kc, vc, bt, cu, sl = b.args()
    o, lse = b.run(mask="window", window=130, n_sink=4)
    od, ld = decode_paged_window(q, kc, vc, bt, sl, b.max_len, window=130, n_sink=4, sinks=b.sinks.cuda())
    b.check(od, ld, mask="window", window=130, n_sink=4)
    b.check(o, lse, mask="window", window=130, n_sink=4)
    b.sinks = None
    od, ld = decode_paged(q, kc, vc, bt, sl, b.max_len)
    o, lse = b.run()
    b.check(od, ld), b.check(o, lse)
    b = Batch([40] * 3, [40, 300, 555], 8, 2, 64, 16, 16)
    q, kc, vc, bt, cu, sl = b.args()
    op, lp = prefill_paged(q.view(3, 40, 8, 64).transpose(1, 2).contiguous(), kc, vc, bt, sl, b.max_len)
    b.check(op.transpose(1, 2).reshape(120, 8, 64), lp.transpose(1, 2).reshape(120, 8))
    b.check(*b.run())


def test_two_captured_steps_replay_on_new_lengths():
    """Two graphs captured side by side, each with a workspace of its own pool, replayed in turn with lengths that
    change what is cut where."""
    a, c = Batch([1, 60, 3], [4000, 900, 500], 8, 2, 128, 16, 17), Batch([9, 1], [300, 6000], 4, 4, 64, 32, 18)
    runs = []
    for b in (a, c):
        b.run()
        args = b.args()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, lse = prefill_paged_varlen(*args, b.max_len)
        runs.append((b, args, graph, o, lse))
    for lens in (None, ([2000, 60, 3], [9, 129]), ([1, 850, 499], [250, 5999])):
        for i, (b, args, graph, o, lse) in enumerate(runs):
            if lens:
                b.ctx = lens[i]
                args[5].copy_(torch.tensor(b.ctx, dtype=I32))
        for b, args, graph, o, lse in runs:
            graph.replay()
        torch.cuda.synchronize()
        for b, args, graph, o, lse in runs:
            t = [torch.arange(m) for m in b.ctx]
            b.k = [b.k_cache[b.table[s].long()[t[s] // b.bs], t[s] % b.bs] for s in range(len(b.ctx))]
            b.v = [b.v_cache[b.table[s].long()[t[s] // b.bs], t[s] % b.bs] for s in range(len(b.ctx))]
            b.check(o, lse)


def test_named_stream_and_workspace_bounds():
    b = Batch([1, 90], [3000, 200], 8, 2, 64, 16, 19)
    want = b.run()
    s = torch.cuda.Stream()
    args = b.args()
    n = prefill_paged_varlen_workspace_bytes(64)
    buf = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    got = prefill_paged_varlen(*args, b.max_len, stream=s, workspace=buf[:n])
    s.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert (buf[n:] == 0xA5).all()
    with pytest.raises(AttnError):
        prefill_paged_varlen(*args, b.max_len, workspace=buf[:n - 16])


def test_offsets_past_32_bits():
    """The last rows of a packed tensor and the last blocks of pools of more than 2^31 elements each."""
    Hq, Hkv, d, bs, T, nb = 128, 8, 128, 16, 140_000, 140_000
    b = Batch([10], [40], Hq, Hkv, d, bs, 24)
    q, out = (torch.empty((T, Hq, d), dtype=BF16, device="cuda") for _ in range(2))
    kc, vc = (torch.empty((nb, bs, Hkv, d), dtype=BF16, device="cuda") for _ in range(2))
    assert min(q.numel(), kc.numel()) > 2 ** 31
    q[T - 10:] = b.q.cuda()
    out[T - 11] = 7.0
    table = torch.tensor([[nb - 1, nb - 3, nb - 2]], dtype=I32)
    t = torch.arange(40)
    where = table[0].long()[t // bs].cuda(), (t % bs).cuda()
    kc[where], vc[where] = b.k[0].cuda(), b.v[0].cuda()
    o, lse = prefill_paged_varlen(q, kc, vc, table.cuda(), torch.tensor([T - 10, T], dtype=I32, device="cuda"),
                                  torch.tensor([40], dtype=I32, device="cuda"), 40, out=out)
    b.check(o[T - 10:], lse[T - 10:])
    assert (out[T - 11] == 7).all()


@pytest.mark.parametrize("n,ctx,Hq,Hkv,d", [([300, 200], [2000, 900], 8, 2, 128), ([1, 3, 8], [3000, 700, 5000], 8, 2, 64),
                                            ([1, 150, 2], [9000, 4000, 300], 16, 2, 128)])
def test_an_expired_wait_is_reported_and_ends(monkeypatch, n, ctx, Hq, Hkv, d):
    """A one-cycle budget lets the pipeline's waits give up: the call comes back with the timeout bit, NaN rows where
    work was left, writes nothing else, and the next call is right. The budget counts from behind the first try, which
    the hardware may itself hold for longer than a short item's copies take: where the few tiles a multiprocessor has
    come through on first tries alone, no bit is set and every row has to be right."""
    b = Batch(n, ctx, Hq, Hkv, d, 16, 21)
    status = torch.zeros(1, dtype=I32, device="cuda")
    q, *rest = b.args()
    q = torch.cat([q, q[:7]])
    out = torch.full((b.T + 7, Hq, d), 5.0, dtype=BF16, device="cuda")
    lse = torch.full((b.T + 7, Hq), 5.0, device="cuda")
    monkeypatch.setenv("ATTN_WAIT_BUDGET_CYCLES", "1")
    prefill_paged_varlen(q, *rest, b.max_len, out=out, lse=lse, status=status)
    torch.cuda.synchronize()
    monkeypatch.delenv("ATTN_WAIT_BUDGET_CYCLES")
    if int(status.item()) == 0:
        assert max(ctx) * Hkv <= 10000  # the largest batch has more tiles a multiprocessor than its ring holds
        b.check(out[:b.T], lse[:b.T])
    else:
        assert int(status.item()) == 0x2 and torch.isnan(out[:b.T].float()).any()
    assert not (out[:b.T] == 5).all(-1).any() and (out[b.T:] == 5).all() and (lse[b.T:] == 5).all()
    b.run_and_check()


def test_scores_without_a_finite_value():
    """An infinite key element makes whole scores -inf: such keys weigh nothing, the others are as without them."""
    b = Batch([3, 70], [400, 300], 4, 2, 64, 16, 22)
    b.q = b.q.abs() + 0.125
    for k in b.k:
        k[:256 if len(k) > 300 else 140, :, 0] = -math.inf
    for s, c in enumerate(b.ctx):
        t = torch.arange(c)
        b.k_cache[b.table[s].long()[t // 16], t % 16] = b.k[s]
    status = torch.zeros(1, dtype=I32, device="cuda")
    o, lse = b.run(status=status)
    assert int(status.item()) == 0
    for s, (n, c) in enumerate(zip(b.n, b.ctx)):
        gone = 256 if c > 300 else 140
        cut = Batch.__new__(Batch)
        cut.__dict__.update(b.__dict__)
        # the same rows against the keys that are left
        cut.n, cut.ctx, cut.k, cut.v = [n], [c - gone], [b.k[s][gone:]], [b.v[s][gone:]]
        cut.q, cut.cu = b.q[int(b.cu[s]):int(b.cu[s + 1])], torch.tensor([0, n])
        r = slice(int(b.cu[s]), int(b.cu[s + 1]))
        cut.check(o[r], lse[r])


def test_refusals():
    b = Batch([2, 3], [20, 30], 4, 2, 64, 16, 20)
    q, kc, vc, bt, cu, sl = b.args()
    ok = dict(q=q, k_cache=kc, v_cache=vc, block_table=bt, cu_q=cu, seq_lens=sl, max_seq_len=30)
    prefill_paged_varlen(*ok.values())
    for kw, err in [(dict(q=q.cpu()), ValueError), (dict(q=q.float()), TypeError), (dict(q=q[:, :3]), ValueError),
                    (dict(q=q.transpose(0, 1)), ValueError), (dict(v_cache=vc[:-1]), ValueError), (dict(k_cache=kc[..., :32]), ValueError),
                    (dict(cu_q=cu[:-1]), ValueError), (dict(cu_q=cu.long()), TypeError), (dict(seq_lens=sl[:1]), ValueError),
                    (dict(block_table=bt[0]), ValueError), (dict(max_seq_len=10 ** 5), AttnError), (dict(mask="none"), ValueError),
                    (dict(mask="window"), AttnError), (dict(n_sink=2), AttnError), (dict(scale=-1.0), AttnError),
                    (dict(sinks=torch.zeros(3, device="cuda")), ValueError), (dict(out=q[:2]), ValueError),
                    (dict(lse=torch.zeros((5, 3), device="cuda")), ValueError), (dict(status=torch.zeros(1, device="cuda")), TypeError),
                    (dict(workspace=torch.zeros(16)), ValueError)]:
        a = dict(ok, **kw)
        with pytest.raises(err):
            prefill_paged_varlen(*[a.pop(k) for k in list(ok)], **a)
