"""qk_norm_rope, its paged form and its backward pass against the formulas in
64 bits.

Tolerances, per element, derived from the roundings: the output is rounded to
bf16 once, at most 2^-8 of its value. Before that the chain in fp32 is the mean
of squares (8 products and sums in a lane, up to 4 sums over lanes: 12
roundings, halved by the square root), its scaling and eps (2), the reciprocal
root (2 units), two products and a rotation of 3 roundings: under 16 roundings
of 2^-24, so 2^-20 of |a cos| + |b sin| at most; 2^-19 is allowed. The backward
pass adds the dot product g n (12 roundings more), two products and a
difference: 2^-18 of r (|g| + |n| mean |g n|). A weight gradient is a sum of
that kind: a thread's 4 rows, 2 lane groups, 8 warps, 32 + 32 partial sums make
under 80 roundings, plus the terms' own 2^-18: 2^-17 of the sum of |dy n|.
"""

import math

import pytest
import torch

from exact_softmax_attention_causal_b200 import (AttnError, qk_norm_rope, qk_norm_rope_backward,
                                                  qk_norm_rope_backward_workspace_bytes, qk_norm_rope_paged)

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
HALF_STEP = 2.0 ** -8
EPS = 1e-6


def _angles64(max_pos, rd):
    inv = 10000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64) / rd)
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def _pairs(x, rd, inter):
    return (x[..., 0:rd:2], x[..., 1:rd:2]) if inter else (x[..., :rd // 2], x[..., rd // 2:rd])


def _join(u, w, rest, inter):
    both = torch.stack([u, w], -1).flatten(-2) if inter else torch.cat([u, w], -1)
    return torch.cat([both, rest], -1)


def turn(x, cos, sin, inter):
    """x [B, N, H, d]; cos, sin [B, N, rd / 2]."""
    rd = 2 * cos.shape[-1]
    a, b = _pairs(x, rd, inter)
    c, s = cos[:, :, None], sin[:, :, None]
    return _join(a * c - b * s, b * c + a * s, x[..., rd:], inter)


def turn_abs(x, cos, sin, inter):
    rd = 2 * cos.shape[-1]
    a, b = _pairs(x.abs(), rd, inter)
    c, s = cos[:, :, None].abs(), sin[:, :, None].abs()
    return _join(a * c + b * s, b * c + a * s, x[..., rd:].abs(), inter)


def norm(x, w):
    if w is None:
        return x
    return x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w


def _case(B, N, Hq, Hkv, d, seed=0, fused=True, w=torch.float32):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((B, N, Hq + 2 * Hkv, d), generator=g).to(BF16)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    if not fused:  # another order of axes, and a gap between heads
        q = q.transpose(1, 2).contiguous().transpose(1, 2)
        pad = torch.zeros((B, N, 2 * Hkv, d), dtype=BF16)
        pad[:, :, ::2] = k
        k, v = pad[:, :, ::2], v.transpose(0, 1).contiguous().transpose(0, 1)
    wq, wk = (None, None) if w is None else ((1 + 0.3 * torch.randn(d, generator=g)).to(w) for _ in range(2))
    return q, k, v, wq, wk


def _cuda(x):
    if x is None:
        return None
    out = torch.empty_strided(x.size(), x.stride(), dtype=x.dtype, device="cuda")
    return out.copy_(x)


def _d(x):
    return None if x is None else x.double()


def _near(got, ref, slack, what):
    got = got.double().cpu()
    bad = (got - ref).abs() > HALF_STEP * ref.abs() + slack
    assert not bad.any(), (what, int(bad.sum()), float((got - ref).abs().max()))


def _positions(kind, B, N, max_pos, seed=1):
    if kind is None:
        return None
    return torch.randint(0, max_pos, (B, N), generator=torch.Generator().manual_seed(seed)).int()


SHAPES = [(1, 1, 1, 1, 64), (1, 1, 8, 2, 128), (2, 5, 3, 1, 64), (1, 130, 5, 5, 128), (3, 33, 9, 3, 64), (2, 64, 32, 8, 128)]


@pytest.mark.parametrize("B,N,Hq,Hkv,d", SHAPES)
@pytest.mark.parametrize("rd,inter,w,pos,fused", [(None, False, torch.float32, None, True),
                                                  (16, True, torch.float32, "random", False),
                                                  (48, False, BF16, "random", True), (32, True, None, None, True),
                                                  (None, True, BF16, None, False), (64, False, None, "random", False)])
def test_forward(B, N, Hq, Hkv, d, rd, inter, w, pos, fused):
    rd = d if rd is None else rd
    max_pos = N + 300
    q, k, v, wq, wk = _case(B, N, Hq, Hkv, d, N, fused, w)
    cos, sin = _angles64(max_pos, rd)
    p = _positions(pos, B, N, max_pos)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = qk_norm_rope(_cuda(q), _cuda(k), _cuda(v), _cuda(wq), _cuda(wk), cos.cuda(), sin.cuda(), positions=_cuda(p),
                       eps=EPS, interleaved=inter, status=status)
    at = torch.arange(N).expand(B, N) if p is None else p.long()
    c, s = cos.double()[at], sin.double()[at]
    for x, wt, y, name in ((q, wq, got[0], "q"), (k, wk, got[1], "k")):
        n = norm(x.double(), _d(wt))
        assert y.is_contiguous() and y.shape == (B, x.shape[2], N, d)
        _near(y.transpose(1, 2), turn(n, c, s, inter), 2.0 ** -19 * turn_abs(n, c, s, inter), name)
    assert torch.equal(got[2].cpu(), v.transpose(1, 2))
    assert int(status.item()) == 0


def _slots(T, num_slots, seed):
    return torch.randperm(num_slots, generator=torch.Generator().manual_seed(seed))[:T].int()


@pytest.mark.parametrize("T,Hq,Hkv,d,bs", [(1, 4, 1, 64, 16), (1, 32, 8, 128, 16), (77, 6, 2, 128, 64), (300, 16, 2, 64, 1),
                                           (65, 5, 5, 64, 128)])
@pytest.mark.parametrize("rd,inter,w", [(64, False, torch.float32), (32, True, BF16), (48, False, None)])
def test_paged(T, Hq, Hkv, d, bs, rd, inter, w):
    q, k, v, wq, wk = _case(1, T, Hq, Hkv, d, T, True, w)
    cos, sin = _angles64(2000, rd)
    pos = _positions("random", 1, T, 2000)
    nb = -(-T // bs) + 3
    slots = _slots(T, nb * bs, 3)
    if T > 2:
        slots[T // 2] = -1  # a row of padding
    g = torch.Generator().manual_seed(8)
    kc, vc = (torch.randn((nb, bs, Hkv, d), generator=g).to(BF16) for _ in range(2))
    kd, vd = kc.cuda(), vc.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = qk_norm_rope_paged(_cuda(q)[0], _cuda(k)[0], _cuda(v)[0], _cuda(wq), _cuda(wk), cos.cuda(), sin.cuda(),
                            pos[0].cuda(), slots.cuda(), kd, vd, eps=EPS, interleaved=inter, status=status)
    c, s = cos.double()[pos.long()], sin.double()[pos.long()]
    n = norm(q.double(), _d(wq))
    _near(qo, turn(n, c, s, inter)[0], 2.0 ** -19 * turn_abs(n, c, s, inter)[0], "q")
    n = norm(k.double(), _d(wk))
    y, slack = turn(n, c, s, inter)[0], 2.0 ** -19 * turn_abs(n, c, s, inter)[0]
    real = slots >= 0
    flat_k, flat_v = kd.cpu().view(-1, Hkv, d), vd.cpu().view(-1, Hkv, d)
    _near(flat_k[slots[real].long()], y[real], slack[real], "k")
    assert torch.equal(flat_v[slots[real].long()], v[0][real])
    other = torch.ones(nb * bs, dtype=torch.bool)
    other[slots[real].long()] = False
    assert torch.equal(flat_k[other], kc.view(-1, Hkv, d)[other])
    assert torch.equal(flat_v[other], vc.view(-1, Hkv, d)[other])
    assert int(status.item()) == 0


def backward_ref(x, w, dz, cos, sin, inter):
    """(dx, dw, slack of dx, slack of dw); dz [B, N, H, d]."""
    dy, ay = turn(dz, cos, -sin, inter), turn_abs(dz, cos, sin, inter)
    if w is None:
        return dy, None, 2.0 ** -19 * ay, None
    r = 1 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
    n, g, ag = x * r, dy * w, ay * w.abs()
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    slack = 2.0 ** -18 * r * (ag + n.abs() * (ag * n.abs()).mean(-1, keepdim=True))
    return dx, (dy * n).sum((0, 1, 2)), slack, 2.0 ** -17 * (ay * n.abs()).sum((0, 1, 2))


@pytest.mark.parametrize("B,N,Hq,Hkv,d", SHAPES)
@pytest.mark.parametrize("rd,inter,w,pos,fused", [(None, False, torch.float32, None, True), (32, True, BF16, "random", False),
                                                  (48, False, None, None, True)])
def test_backward(B, N, Hq, Hkv, d, rd, inter, w, pos, fused):
    rd = d if rd is None else rd
    q, k, v, wq, wk = _case(B, N, Hq, Hkv, d, N + 1, fused, w)
    g = torch.Generator().manual_seed(4)
    dz = [torch.randn((B, H, N, d), generator=g).to(BF16) for H in (Hq, Hkv, Hkv)]
    cos, sin = _angles64(N + 50, rd)
    p = _positions(pos, B, N, N + 50)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = {}
    if not fused:
        kw = dict(dq=torch.empty((B, Hq, N, d), dtype=BF16, device="cuda").transpose(1, 2))
    args = [_cuda(t) for t in (q, k, wq, wk, cos, sin, *dz)]
    dq, dk, dv, dwq, dwk = qk_norm_rope_backward(*args, positions=_cuda(p), eps=EPS, interleaved=inter, status=status, **kw)
    again = qk_norm_rope_backward(*args, positions=_cuda(p), eps=EPS, interleaved=inter, **kw)
    at = torch.arange(N).expand(B, N) if p is None else p.long()
    c, s = cos.double()[at], sin.double()[at]
    for x, wt, z, dx, dw, name in ((q, wq, dz[0], dq, dwq, "q"), (k, wk, dz[1], dk, dwk, "k")):
        rx, rw, sx, sw = backward_ref(x.double(), _d(wt), z.double().transpose(1, 2), c, s, inter)
        _near(dx, rx, sx, "d" + name)
        if w is not None:
            assert dw.dtype == torch.float32
            assert not ((dw.double().cpu() - rw).abs() > sw).any(), name
    assert torch.equal(dv.cpu(), dz[2].transpose(1, 2))
    assert int(status.item()) == 0
    if w is None:
        assert dwq is None and dwk is None
    for a, b in zip((dq, dk, dv, dwq, dwk), again):
        assert a is None or torch.equal(a, b)  # the same bits on every run


def test_gradients_against_differences():
    """Central differences of the 64-bit forward along a random direction against the kernel's gradients; the
    gradients' bf16 rounding, 2^-8 of each, is what may be off."""
    B, N, Hq, Hkv, d, rd = 1, 3, 2, 1, 64, 48
    q, k, v, wq, wk = _case(B, N, Hq, Hkv, d, 11)
    g = torch.Generator().manual_seed(2)
    dz = [torch.randn((B, H, N, d), generator=g).to(BF16) for H in (Hq, Hkv, Hkv)]
    cos, sin = _angles64(N, rd)
    dq, dk, dv, dwq, dwk = [t.double().cpu() for t in qk_norm_rope_backward(
        *[_cuda(t) for t in (q, k, wq, wk, cos, sin, *dz)], eps=EPS)]
    c, s = cos.double()[None], sin.double()[None]
    for x, w, z, dx, dw in ((q, wq, dz[0], dq, dwq), (k, wk, dz[1], dk, dwk)):
        x, w, z = x.double(), w.double(), z.double().transpose(1, 2)
        ux, uw = torch.randn(x.shape, generator=g, dtype=torch.float64), torch.randn(d, generator=g, dtype=torch.float64)

        def loss(h):
            return (turn(norm(x + h * ux, w + h * uw), c, s, False) * z).sum()

        h = 1e-5
        diff = (loss(h) - loss(-h)) / (2 * h)
        got = (dx * ux).sum() + (dw * uw).sum()
        slack = (2.0 ** -8 + 2.0 ** -12) * (dx * ux).abs().sum() + 2.0 ** -17 * (dw * uw).abs().sum() * d + 1e-6
        assert abs(float(got - diff)) <= float(slack)


def test_bad_positions_and_slots_are_flagged_and_write_nothing_else():
    T, Hq, Hkv, d = 6, 4, 2, 64
    q, k, v, wq, wk = [_cuda(t) for t in _case(1, T, Hq, Hkv, d)]
    cos, sin = [t.cuda() for t in _angles64(50, d)]
    kc = torch.zeros((4, 16, Hkv, d), dtype=BF16, device="cuda")
    vc = torch.zeros_like(kc)
    for pos, slots, bad_q in [([0, 1, 50, 3, 4, 5], [0, 1, 2, 3, 4, 5], [2]), ([0, -1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5], [1]),
                              ([0, 1, 2, 3, 4, 5], [0, 1, 64, 3, -2, 5], [])]:
        kc.zero_(), vc.zero_()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        p, s = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in (pos, slots))
        out = qk_norm_rope_paged(q[0], k[0], v[0], wq, wk, cos, sin, p, s, kc, vc, status=status)
        assert int(status.item()) == 1
        nan = torch.isnan(out.float()).flatten(1).all(1).tolist()
        assert [i for i in range(T) if nan[i]] == bad_q
        written = kc.view(-1, Hkv * d).ne(0).any(1).nonzero().flatten().tolist()
        assert written == [s for i, s in enumerate(slots) if 0 <= s < 64 and i not in bad_q]
        assert written == vc.view(-1, Hkv * d).ne(0).any(1).nonzero().flatten().tolist()
    pos = torch.zeros((1, T), dtype=torch.int32, device="cuda")
    pos[0, 3] = 99
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    yq, yk, yv = qk_norm_rope(q, k, v, wq, wk, cos, sin, positions=pos, status=status)
    assert int(status.item()) == 1
    assert torch.isnan(yq[:, :, 3].float()).all() and torch.isfinite(yq[:, :, :3].float()).all()
    assert torch.equal(yv, v.transpose(1, 2))


def test_infinities_stay_in_their_head():
    q, k, v, _, _ = _case(1, 4, 2, 1, 64)
    q, k = q.clone(), k.clone()
    q[0, 1, 0, 50] = math.inf  # past the turned part: goes through, without touching it
    q[0, 2, 1, 3] = math.nan
    cos, sin = _angles64(4, 32)
    y, _, _ = qk_norm_rope(_cuda(q), _cuda(k), _cuda(v), None, None, cos.cuda(), sin.cuda())
    y = y.cpu().float()
    assert y[0, 0, 1, 50] == math.inf and torch.isfinite(y[0, 0, 1, :50]).all()
    assert torch.isnan(y[0, 1, 2, [3, 19]]).all() and torch.isnan(y).sum() == 2


def test_capture_streams_and_guards():
    B, N, Hq, Hkv, d = 2, 40, 8, 2, 128
    q, k, v, wq, wk = [_cuda(t) for t in _case(B, N, Hq, Hkv, d)]
    cos, sin = [t.cuda() for t in _angles64(N, d)]
    want = qk_norm_rope(q, k, v, wq, wk, cos, sin)
    dz = [torch.randn_like(t) for t in want]
    wantg = qk_norm_rope_backward(q, k, wq, wk, cos, sin, *dz)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = qk_norm_rope(q, k, v, wq, wk, cos, sin, stream=s)
    gotg = qk_norm_rope_backward(q, k, wq, wk, cos, sin, *dz, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want + wantg, got + gotg))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = qk_norm_rope(q, k, v, wq, wk, cos, sin)
        capg = qk_norm_rope_backward(q, k, wq, wk, cos, sin, *dz)
    q.mul_(-0.5)
    graph.replay()
    want = qk_norm_rope(q, k, v, wq, wk, cos, sin)
    wantg = qk_norm_rope_backward(q, k, wq, wk, cos, sin, *dz)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want + wantg, cap + capg))
    # the workspace is used up to its stated size and not beyond
    n = qk_norm_rope_backward_workspace_bytes(B, N, Hq, Hkv, d)
    buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    qk_norm_rope_backward(q, k, wq, wk, cos, sin, *dz, workspace=buf[:n])
    assert (buf[n:] == 0xA5).all()
    with pytest.raises(AttnError):
        qk_norm_rope_backward(q, k, wq, wk, cos, sin, *dz, workspace=buf[:n - 16])


def test_offsets_past_32_bits():
    """Tensors and a pool of more than 2^31 elements: their last rows."""
    N, Hq, Hkv, d, bs = 140_000, 120, 4, 128, 16
    qkv = torch.empty((1, N, Hq + 2 * Hkv, d), dtype=BF16, device="cuda")
    assert qkv.numel() > 2 ** 31 and N * Hq * d > 2 ** 31
    small = _case(1, 8, Hq, Hkv, d)
    qkv[:, N - 8:] = torch.cat([_cuda(t) for t in small[:3]], 2)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    wq, wk = _cuda(small[3]), _cuda(small[4])
    cos, sin = [t.cuda() for t in _angles64(N, d)]
    pos = torch.arange(N - 8, N, dtype=torch.int32, device="cuda")
    want = qk_norm_rope(q[:, N - 8:].contiguous(), k[:, N - 8:], v[:, N - 8:], wq, wk, cos, sin, positions=pos[None])
    got = qk_norm_rope(q, k, v, wq, wk, cos, sin)
    assert all(torch.equal(a, b[:, :, N - 8:]) for a, b in zip(want, got))
    dz = [torch.empty_like(t) for t in got]
    for t in dz:
        t[:, :, N - 8:] = torch.randn(t[:, :, N - 8:].shape, device="cuda").to(BF16)
    del got
    # without weights: a weight's gradient would sum the rows nobody filled
    wantg = qk_norm_rope_backward(q[:, N - 8:], k[:, N - 8:], None, None, cos, sin, *[t[:, :, N - 8:].contiguous() for t in dz],
                                  positions=pos[None])
    gotg = qk_norm_rope_backward(q, k, None, None, cos, sin, *dz)
    assert all(torch.equal(a, b[:, N - 8:]) for a, b in zip(wantg[:3], gotg[:3]))
    del gotg, dz
    nb = 270_000
    kc, vc = (torch.zeros((nb, bs, Hkv, d), dtype=BF16, device="cuda") for _ in range(2))
    assert kc.numel() > 2 ** 31
    slots = torch.arange(nb * bs - 8, nb * bs, dtype=torch.int32, device="cuda")
    qk_norm_rope_paged(q[0, N - 8:], k[0, N - 8:], v[0, N - 8:], wq, wk, cos, sin, pos, slots, kc, vc)
    assert torch.equal(kc.view(-1, Hkv, d)[-8:], want[1][0].transpose(0, 1)) and torch.equal(vc.view(-1, Hkv, d)[-8:], v[0, N - 8:])
    assert not kc.view(-1, Hkv, d)[:8].any() and not kc.view(-1, Hkv, d)[-9].any()


def test_an_empty_step_does_nothing():
    q, k, v, wq, wk = [_cuda(t) for t in _case(1, 1, 4, 2, 64)]
    cos, sin = [t.cuda() for t in _angles64(4, 64)]
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    kc = torch.zeros((1, 16, 2, 64), dtype=BF16, device="cuda")
    out = qk_norm_rope_paged(q[0, :0], k[0, :0], v[0, :0], wq, wk, cos, sin, none, none, kc, kc.clone())
    assert out.shape == (0, 4, 64) and not kc.any()


def test_refusals():
    B, N, Hq, Hkv, d = 1, 4, 4, 2, 64
    q, k, v, wq, wk = [_cuda(t) for t in _case(B, N, Hq, Hkv, d)]
    cos, sin = [t.cuda() for t in _angles64(N, d)]
    ok = dict(q=q, k=k, v=v, q_weight=wq, k_weight=wk, cos=cos, sin=sin)
    qk_norm_rope(*ok.values())
    small = torch.randn((B, N, Hq, 96), device="cuda").to(BF16)
    odd = torch.zeros(B * N * Hq * d + 8, dtype=BF16, device="cuda")[1:1 + B * N * Hq * d].view(B, N, Hq, d)
    for kw, err in [(dict(q=q.cpu()), ValueError), (dict(q=q.float()), TypeError), (dict(k=k[:, :3]), ValueError),
                    (dict(v=v[..., :32]), ValueError), (dict(q=q.transpose(2, 3).contiguous().transpose(2, 3)), ValueError),
                    (dict(q_weight=None), ValueError), (dict(k_weight=wk.to(BF16)), TypeError),
                    (dict(q_weight=wq.half(), k_weight=wk.half()), TypeError), (dict(cos=cos[:3], sin=sin[:3]), AttnError),
                    (dict(cos=cos[:, :20].contiguous(), sin=sin[:, :20].contiguous()), AttnError), (dict(sin=sin[:2]), ValueError),
                    (dict(q=small, k=small[:, :, :2], v=small[:, :, :2], q_weight=None, k_weight=None), AttnError),
                    (dict(q=odd), AttnError), (dict(eps=-1.0), AttnError), (dict(eps=float("nan")), AttnError),
                    (dict(positions=torch.zeros((B, N), device="cuda")), TypeError),
                    (dict(positions=torch.zeros((B, N + 1), dtype=torch.int32, device="cuda")), ValueError),
                    (dict(q_out=torch.empty((B, N, Hq, d), dtype=BF16, device="cuda")[:, :2]), ValueError)]:
        a = dict(ok, **kw)
        with pytest.raises(err):
            qk_norm_rope(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("q_weight"), a.pop("k_weight"), a.pop("cos"), a.pop("sin"), **a)
    dz = [t.transpose(1, 2).contiguous() for t in (q, k, v)]
    with pytest.raises(ValueError):  # two tokens' gradients may not land in one place
        qk_norm_rope_backward(q, k, wq, wk, cos, sin, *dz, dq=torch.empty((B, 1, Hq, d), dtype=BF16, device="cuda").expand(B, N, Hq, d))
    with pytest.raises(ValueError):
        qk_norm_rope_backward(q, k, wq, wk, cos, sin, dz[0].transpose(1, 2), dz[1], dz[2])
