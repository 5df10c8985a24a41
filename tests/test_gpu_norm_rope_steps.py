"""qk_norm_rope, its paged form and its backward pass at sizes where a CTA takes
many steps: chunks of 4 heads of a tile of tokens (16 tokens at d = 128, 32 at
d = 64), from q to k to v and on to the next tile, each step's rows copied ahead
of it.

Tolerances of elements are those derived in test_gpu_norm_rope.py. A weight's
gradient is a sum in fp32: 4 rows of a chunk, then a thread's chunks one after
another, 2 or 4 lane groups, 8 warps, the CTAs' sums by 32 warps, and those 32.
With S steps a thread that are S + 4 + 4 + 8 + ceil(CTAs / 32) + 32 roundings of
2^-24 of the sum of |dy n| at most, besides the terms' own 2^-18.
"""

import pytest
import torch

from exact_softmax_attention_causal_b200 import (qk_norm_rope, qk_norm_rope_backward,
                                                  qk_norm_rope_backward_workspace_bytes, qk_norm_rope_paged)
from test_gpu_norm_rope import BF16, EPS, HALF_STEP, _angles64, _case, _cuda, _d, _positions, norm, turn, turn_abs

pytestmark = pytest.mark.gpu


def _tiles(tokens, d):
    return -(-tokens // (2048 // d))


def _chunks(Hq, Hkv):
    return -(-Hq // 4) + 2 * -(-Hkv // 4)


def _forward_steps(tokens, Hq, Hkv, d):
    """Chunks that a CTA of the forward pass goes through, at least."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    parts = min(-(-8 * sms // _tiles(tokens, d)), _chunks(Hq, Hkv))
    return _chunks(Hq, Hkv) // parts


def _near(got, ref, slack, what):
    bad = ~((got.double() - ref).abs() <= HALF_STEP * ref.abs() + slack)
    assert not bad.any(), (what, int(bad.sum()), float((got.double() - ref).abs().max()))


FORMS = [(128, False, torch.float32, None), (48, True, BF16, "random"), (64, False, None, "random")]


def _inputs(B, N, Hq, Hkv, d, rd, w, pos, seed):
    rd = min(rd, d)
    x = [_cuda(t) for t in _case(B, N, Hq, Hkv, d, seed, True, w)]
    cos, sin = (t.cuda() for t in _angles64(N + 60, rd))
    p = _cuda(_positions(pos, B, N, N + 60))
    at = torch.arange(N, device="cuda").expand(B, N) if p is None else p.long()
    return x, cos, sin, p, cos.double()[at], sin.double()[at]


@pytest.mark.parametrize("B,N,Hq,Hkv,d", [(2, 2051, 32, 8, 128), (3, 6667, 9, 3, 128), (1, 40001, 9, 3, 64), (2, 4099, 16, 16, 64)])
@pytest.mark.parametrize("rd,inter,w,pos", FORMS)
def test_forward(B, N, Hq, Hkv, d, rd, inter, w, pos):
    assert _forward_steps(B * N, Hq, Hkv, d) >= 2
    (q, k, v, wq, wk), cos, sin, p, c, s = _inputs(B, N, Hq, Hkv, d, rd, w, pos, N)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = qk_norm_rope(q, k, v, wq, wk, cos, sin, positions=p, eps=EPS, interleaved=inter, status=status)
    for x, wt, y, name in ((q, wq, got[0], "q"), (k, wk, got[1], "k")):
        n = norm(x.double(), _d(wt))
        _near(y.transpose(1, 2), turn(n, c, s, inter), 2.0 ** -19 * turn_abs(n, c, s, inter), name)
    assert torch.equal(got[2], v.transpose(1, 2))
    assert int(status.item()) == 0


@pytest.mark.parametrize("T,Hq,Hkv,d,bs", [(4099, 32, 8, 128, 16), (20011, 9, 3, 128, 64), (8191, 64, 8, 64, 64), (40001, 5, 5, 64, 1)])
@pytest.mark.parametrize("rd,inter,w,pos", FORMS)
def test_paged(T, Hq, Hkv, d, bs, rd, inter, w, pos):
    assert _forward_steps(T, Hq, Hkv, d) >= 2
    (q, k, v, wq, wk), cos, sin, p, c, s = _inputs(1, T, Hq, Hkv, d, rd, w, "random", T)
    nb = -(-T // bs) + 5
    g = torch.Generator("cuda").manual_seed(T)
    slots = torch.randperm(nb * bs, generator=g, device="cuda")[:T].int()
    slots[torch.randperm(T, generator=g, device="cuda")[:T // 9]] = -1  # padding, in no order
    kc, vc = (torch.randn((nb, bs, Hkv, d), generator=g, device="cuda").to(BF16) for _ in range(2))
    k0, v0 = kc.clone().view(-1, Hkv, d), vc.clone().view(-1, Hkv, d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = qk_norm_rope_paged(q[0], k[0], v[0], wq, wk, cos, sin, p[0], slots, kc, vc, eps=EPS, interleaved=inter, status=status)
    n = norm(q.double(), _d(wq))
    _near(qo, turn(n, c, s, inter)[0], 2.0 ** -19 * turn_abs(n, c, s, inter)[0], "q")
    n = norm(k.double(), _d(wk))
    real = slots >= 0
    at = slots[real].long()
    kc, vc = kc.view(-1, Hkv, d), vc.view(-1, Hkv, d)
    _near(kc[at], turn(n, c, s, inter)[0][real], 2.0 ** -19 * turn_abs(n, c, s, inter)[0][real], "k")
    assert torch.equal(vc[at], v[0][real])
    other = torch.ones(nb * bs, dtype=torch.bool, device="cuda")
    other[at] = False
    assert torch.equal(kc[other], k0[other]) and torch.equal(vc[other], v0[other])
    assert int(status.item()) == 0


@pytest.mark.parametrize("B,N,Hq,Hkv,d", [(2, 2051, 32, 8, 128), (3, 6667, 9, 3, 128), (1, 12345, 9, 3, 64), (2, 4099, 32, 8, 64),
                                          (5, 2477, 4, 4, 128)])
@pytest.mark.parametrize("rd,inter,w,pos", FORMS)
def test_backward(B, N, Hq, Hkv, d, rd, inter, w, pos):
    (q, k, v, wq, wk), cos, sin, p, c, s = _inputs(B, N, Hq, Hkv, d, rd, w, pos, N + 1)
    ctas = qk_norm_rope_backward_workspace_bytes(B, N, Hq, Hkv, d) // (8 * d)
    tiles, turned, copied = _tiles(B * N, d), -(-Hq // 4) + -(-Hkv // 4), -(-Hkv // 4)
    assert tiles * (turned + copied) >= 4 * ctas  # steps
    # a CTA's share is even in tensor rows moved, 3 for a chunk of q or k and 2 for one of v
    steps = tiles * (3 * turned + 2 * copied) / (3 * ctas) + 2
    g = torch.Generator("cuda").manual_seed(4)
    dz = [torch.randn((B, H, N, d), generator=g, device="cuda").to(BF16) for H in (Hq, Hkv, Hkv)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (q, k, wq, wk, cos, sin, *dz)
    got = qk_norm_rope_backward(*args, positions=p, eps=EPS, interleaved=inter, status=status)
    again = qk_norm_rope_backward(*args, positions=p, eps=EPS, interleaved=inter)
    for x, wt, z, dx, dw, name in ((q, wq, dz[0], got[0], got[3], "q"), (k, wk, dz[1], got[1], got[4], "k")):
        x, z = x.double(), z.double().transpose(1, 2)
        dy, ay = turn(z, c, -s, inter), turn_abs(z, c, s, inter)
        if wt is None:
            _near(dx, dy, 2.0 ** -19 * ay, "d" + name)
            assert dw is None
            continue
        r = 1 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
        n, gw, aw = x * r, dy * wt.double(), ay * wt.double().abs()
        ref = r * (gw - n * (gw * n).mean(-1, keepdim=True))
        _near(dx, ref, 2.0 ** -18 * r * (aw + n.abs() * (aw * n.abs()).mean(-1, keepdim=True)), "d" + name)
        total = (ay * n.abs()).sum((0, 1, 2))
        slack = (2.0 ** -18 + (steps + 48 + ctas / 32) * 2.0 ** -24) * total
        assert ((dw.double() - (dy * n).sum((0, 1, 2))).abs() <= slack).all(), name
    assert torch.equal(got[2], dz[2].transpose(1, 2))
    assert int(status.item()) == 0
    for a, b in zip(got, again):
        assert a is None or torch.equal(a, b)  # the same bits on every run


def test_bad_positions_among_many_steps():
    """One token out of range: its rows and the weights' gradients, and nothing else."""
    B, N, Hq, Hkv, d = 2, 4099, 8, 4, 128
    (q, k, v, wq, wk), cos, sin, p, c, s = _inputs(B, N, Hq, Hkv, d, d, torch.float32, "random", 5)
    dz = [torch.ones((B, H, N, d), device="cuda", dtype=BF16) for H in (Hq, Hkv, Hkv)]
    good = qk_norm_rope_backward(q, k, wq, wk, cos, sin, *dz, positions=p, eps=EPS)
    p[1, 3000] = N + 60
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = qk_norm_rope_backward(q, k, wq, wk, cos, sin, *dz, positions=p, eps=EPS, status=status)
    assert int(status.item()) == 1
    for a, b in zip(got[:2], good[:2]):
        assert torch.isnan(a[1, 3000].float()).all()
        a, b = a.clone(), b.clone()
        a[1, 3000] = b[1, 3000] = 0
        assert torch.equal(a, b)
    assert torch.equal(got[2], good[2]) and torch.isnan(got[3]).all() and torch.isnan(got[4]).all()
