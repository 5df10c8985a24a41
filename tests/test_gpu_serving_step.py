"""The operators around the paged cache run together, as a program uses them.

Serving: each step gives the sequences their blocks and slots (paged_extend),
writes their keys and values into the cache behind norm and rotation
(qk_norm_rope_paged) and attends over it (prefill_paged_varlen); finished
sequences give their blocks back (paged_release) and others take them over.
What a step computes does not depend on how the tokens came, so the reference
is the whole sequence at once: qk_norm_rope gives the same bits as the cache
holds, and softmax attention in 64 bits over them the output.

Training: norm and rotation, attention, and both backward passes, against
automatic differentiation in 64 bits.
"""

import math

import pytest
import torch

from exact_softmax_attention_causal_b200 import (paged_extend, paged_release, prefill, prefill_backward,
                                                  prefill_paged_varlen, qk_norm_rope, qk_norm_rope_backward,
                                                  qk_norm_rope_paged)
from parity import assert_grad_parity

pytestmark = pytest.mark.gpu

BF16, I32 = torch.bfloat16, torch.int32
EPS = 1e-6


def _angles(max_pos, rd):
    inv = 10000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64) / rd)
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return ang.cos().float().cuda(), ang.sin().float().cuda()


class Server:
    def __init__(self, B, Hq, Hkv, d, bs, num_blocks, max_len, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        self.g, self.B, self.Hq, self.Hkv, self.d, self.bs, self.num_blocks, self.max_len = g, B, Hq, Hkv, d, bs, num_blocks, max_len
        self.wq, self.wk = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
        self.cos, self.sin = _angles(max_len, d)
        self.lens = torch.zeros(B, dtype=I32, device="cuda")
        self.table = torch.full((B, -(-max_len // bs)), -1, dtype=I32, device="cuda")
        self.free = torch.randperm(num_blocks, device="cuda", generator=g).to(I32)
        self.num_free = torch.tensor([num_blocks], dtype=I32, device="cuda")
        nan = float("nan")
        self.kc = torch.full((num_blocks, bs, Hkv, d), nan, dtype=BF16, device="cuda")
        self.vc = torch.full_like(self.kc, nan)
        self.status = torch.zeros(1, dtype=I32, device="cuda")
        self.past = [[] for _ in range(B)]  # each sequence's projections so far

    def step(self, qkv, new, T, **mask):
        """One step, all in place; qkv [T, Hq + 2 Hkv, d]."""
        Hq, Hkv = self.Hq, self.Hkv
        _, _, cu, pos, slots = paged_extend(self.lens, new, self.table, self.free, self.num_free, self.bs, self.num_blocks,
                                            T, seq_lens_out=self.lens, num_free_out=self.num_free, status=self.status)
        q = qk_norm_rope_paged(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], self.wq, self.wk, self.cos, self.sin,
                               pos, slots, self.kc, self.vc, eps=EPS, status=self.status)
        return prefill_paged_varlen(q, self.kc, self.vc, self.table, cu, self.lens, self.max_len, status=self.status, **mask)

    def draw(self, new, T):
        qkv = torch.randn((T, self.Hq + 2 * self.Hkv, self.d), generator=self.g, device="cuda").to(BF16)
        at = 0
        for b, n in enumerate(new):
            self.past[b].append(qkv[at:at + n].clone())
            at += n
        return qkv

    def check(self, o, lse, new, window=0):
        """The new rows of every sequence against the whole sequence at once."""
        at = 0
        for b, n in enumerate(new):
            if n == 0:
                continue
            x = torch.cat(self.past[b])[None]
            c = x.shape[1]
            q, k, v = qk_norm_rope(x[:, :, :self.Hq], x[:, :, self.Hq:self.Hq + self.Hkv], x[:, :, self.Hq + self.Hkv:], self.wq,
                                   self.wk, self.cos, self.sin, eps=EPS)
            t = torch.arange(c, device="cuda")
            where = self.table[b].long()[t // self.bs], t % self.bs
            assert torch.equal(self.kc[where], k[0].transpose(0, 1)) and torch.equal(self.vc[where], v[0].transpose(0, 1))
            group = self.Hq // self.Hkv
            q64, k64, v64 = q[0, :, c - n:].double(), *(y[0].double().repeat_interleave(group, 0) for y in (k, v))
            scale = 1 / math.sqrt(self.d)
            s = q64 @ k64.transpose(1, 2) * scale
            i, j = torch.arange(c - n, c, device="cuda")[:, None], t[None]
            s = s.masked_fill((j > i) | ((i - j >= window) if window else (j < 0)), -math.inf)
            rl = torch.logsumexp(s, -1)
            p = (s - rl[..., None]).exp()
            ro, spread = p @ v64, p @ v64.abs()
            # the tolerances of the attention by itself, see its tests
            big = (q64.abs() @ k64.abs().transpose(1, 2)).amax(-1) * scale
            so = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -15 + 2.0 ** -17 * big[..., None]) * spread
            got = o[at:at + n].double().transpose(0, 1)
            assert ((got - ro).abs() <= so).all(), (b, float(((got - ro).abs() - so).max()))
            assert ((lse[at:at + n].double().t() - rl).abs() <= 2.0 ** -18 * (big + 1 + rl.abs())).all(), b
            at += n


@pytest.mark.parametrize("Hq,Hkv,d,bs,window", [(8, 2, 128, 16, 0), (16, 2, 64, 64, 0), (8, 8, 64, 16, 90), (6, 2, 128, 32, 40)])
def test_prompts_in_chunks_beside_decoding_sequences(Hq, Hkv, d, bs, window):
    B = 4
    s = Server(B, Hq, Hkv, d, bs, num_blocks=-(-1500 // bs), max_len=700, seed=Hq)
    mask = dict(mask="window", window=window) if window else {}
    # a long prompt in chunks, short ones that decode beside it, one that ends and another in its place
    plan = [[200, 17, 0, 1], [200, 1, 40, 1], [131, 1, 1, 1], [1, 5, 1, 1], "end 1", [1, 300, 1, 1], [1, 1, 3, 1], "end 0", [64, 1, 1, 1]]
    for new in plan:
        if isinstance(new, str):
            gone = int(new[-1])
            fin = torch.zeros(B, dtype=I32, device="cuda")
            fin[gone] = 1
            paged_release(s.lens, fin, s.table, s.free, s.num_free, s.bs, s.num_blocks, seq_lens_out=s.lens,
                          num_free_out=s.num_free, status=s.status)
            s.past[gone] = []
            continue
        T = sum(new) + 9  # padded
        qkv = s.draw(new, T)
        o, lse = s.step(qkv, torch.tensor(new, dtype=I32, device="cuda"), T, **mask)
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0
        s.check(o, lse, new, window)


def test_a_sequence_without_blocks_does_not_disturb_the_others():
    B, new = 3, [30, 500, 20]
    s = Server(B, 8, 2, 64, 16, num_blocks=10, max_len=600, seed=1)
    qkv = s.draw(new, sum(new))
    o, lse = s.step(qkv, torch.tensor(new, dtype=I32, device="cuda"), sum(new))
    torch.cuda.synchronize()
    assert int(s.status.item()) == 1 and s.lens.tolist() == [30, -1, -1]
    s.check(o, lse, [30, 0, 0])
    assert torch.isnan(o[30:].float()).all() and torch.isnan(lse[30:]).all()
    # the failed ones are let go, and the pool is whole again
    paged_release(s.lens, torch.ones(B, dtype=I32, device="cuda"), s.table, s.free, s.num_free, 16, 10, seq_lens_out=s.lens,
                  num_free_out=s.num_free)
    assert s.lens.tolist() == [0, 0, 0] and sorted(s.free.tolist()) == list(range(10))


def test_decode_steps_as_one_graph():
    B, T = 3, 4  # one row of padding
    s = Server(B, 8, 2, 128, 16, num_blocks=60, max_len=250, seed=2)
    start = [100, 1, 60]
    qkv = s.draw(start, sum(start))
    s.step(qkv, torch.tensor(start, dtype=I32, device="cuda"), sum(start))
    buf = torch.zeros((T, 8 + 4, 128), dtype=BF16, device="cuda")
    new = torch.ones(B, dtype=I32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = s.step(buf, new, T)
    for step in range(40):
        # now and then a sequence sits out
        take = [1, 1, 1] if step % 7 else [1, 0, 1]
        new.copy_(torch.tensor(take, dtype=I32))
        buf.copy_(s.draw(take, T))
        graph.replay()
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0
        s.check(o, lse, take)


@pytest.mark.parametrize("Hq,Hkv,d,rd,inter", [(4, 2, 64, 64, False), (8, 2, 128, 64, True)])
def test_training_step(Hq, Hkv, d, rd, inter):
    """Gradients of the projections within what the attention's backward pass is held to (assert_grad_parity: P, dS and
    its outputs are bf16); the reference rounds the rotated q and k as the forward pass does. A weight's gradient sums
    dy n over all rows, dy off by up to 1 % each and independently: 4 standard deviations of that sum are allowed."""
    B, N = 2, 130
    g = torch.Generator().manual_seed(5)
    x = [torch.randn((B, N, H, d), generator=g).to(BF16) for H in (Hq, Hkv, Hkv)]
    w = [1 + 0.2 * torch.randn(d, generator=g) for _ in range(2)]
    d_o = torch.randn((B, Hq, N, d), generator=g).to(BF16)
    cos, sin = _angles(N, rd)
    xc, wc = [t.cuda() for t in x], [t.cuda() for t in w]
    q, k, v = qk_norm_rope(*xc, *wc, cos, sin, eps=EPS, interleaved=inter)
    o, lse = prefill(q, k, v)
    gq, gk, gv = prefill_backward(q, k, v, o, lse, d_o.cuda())
    dq, dk, dv, dwq, dwk = qk_norm_rope_backward(xc[0], xc[1], *wc, cos, sin, gq, gk, gv, eps=EPS, interleaved=inter)

    c, s = cos.double().cpu()[None, :, None], sin.double().cpu()[None, :, None]
    leaves = [t.double().requires_grad_() for t in x]
    weights = [t.double().requires_grad_() for t in w]

    def rotated(t, wt):
        n = t / (t.square().mean(-1, keepdim=True) + EPS).sqrt()
        y = n * wt
        a, b = (y[..., 0:rd:2], y[..., 1:rd:2]) if inter else (y[..., :rd // 2], y[..., rd // 2:rd])
        u, e = a * c - b * s, b * c + a * s
        z = torch.cat([torch.stack([u, e], -1).flatten(-2) if inter else torch.cat([u, e], -1), y[..., rd:]], -1)
        return z + (z.to(BF16).double() - z).detach(), n, y

    q64, nq, yq = rotated(leaves[0], weights[0])
    k64, nk, yk = rotated(leaves[1], weights[1])
    yq.retain_grad(), yk.retain_grad()
    group = Hq // Hkv
    kk, vv = (t.repeat_interleave(group, 2) for t in (k64, leaves[2]))
    sc = torch.einsum("bnhd,bmhd->bhnm", q64, kk) / math.sqrt(d)
    sc = sc.masked_fill(torch.ones(N, N, dtype=torch.bool).triu(1), -math.inf)
    out = torch.einsum("bhnm,bmhd->bhnd", sc.softmax(-1), vv)
    (out * d_o.double()).sum().backward()
    for got, ref, name in ((dq, leaves[0].grad, "dq"), (dk, leaves[1].grad, "dk"), (dv, leaves[2].grad, "dv")):
        assert_grad_parity(got, ref, what=name)
    for got, ref, y, n in ((dwq, weights[0].grad, yq, nq), (dwk, weights[1].grad, yk, nk)):
        spread = (y.grad * n).square().sum((0, 1, 2)).sqrt().detach()
        assert ((got.double().cpu() - ref).abs() <= 0.04 * spread).all()
