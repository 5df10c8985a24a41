"""Operators around the paged cache and the prefill, as cases to measure.

Three groups, each in its plain form (elementary torch operations in 32 bits)
and as the calls a user makes of the package (``own``):

* block tables: ``paged_extend`` gives every sequence the blocks that its new
  tokens need and writes the tokens' positions and slots; ``paged_release``
  returns the blocks of finished sequences.
* query and key norms with the position rotation in the same pass:
  ``qk_norm_rope`` (into the layout of ``prefill``), its backward pass, and
  ``qk_norm_rope_paged``, which writes K and V into the paged cache.
* ``prefill_paged_varlen``: each sequence's own number of new tokens against
  its paged context.
"""

import math

import torch

own = False

_lib = None


def _attn():
    global _lib
    if _lib is None:
        import exact_softmax_attention_causal_b200 as attn

        _lib = attn
    return _lib


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 64 running requests: one new token each, a block for one in sixteen
        dict(name="extend_decode_b64", op="extend", B=64, len_lo=1024, len_hi=32767, new_lo=1, new_hi=1, bs=16,
             max_len=32768, pad=0),
        # a scheduler step that mixes waiting prompts with running requests, padded to a fixed token count
        dict(name="extend_mixed_b512", op="extend", B=512, len_lo=0, len_hi=8192, new_lo=0, new_hi=255, bs=16,
             max_len=16384, pad=777),
        # a third of 512 requests end: their blocks go back
        dict(name="release_b512", op="release", B=512, len_lo=0, len_hi=16384, bs=16, max_len=16384),
        # training: the Llama-3-8B shapes of the prefill, with query and key norms
        dict(name="norm_rope_train", op="norm_rope", B=4, N=4096, Hq=32, Hkv=8, d=128, rd=128, inter=False,
             norm=True, pos=False),
        # the backward pass of the same step
        dict(name="norm_rope_train_bwd", op="norm_rope_bwd", B=4, N=4096, Hq=32, Hkv=8, d=128, rd=128, inter=False,
             norm=True, pos=False),
        # one decode step: 64 tokens, each appended to its own block
        dict(name="norm_rope_append_b64", op="norm_rope_paged", T=64, Hq=32, Hkv=8, d=128, rd=128, inter=False,
             norm=True, bs=16, pad=0),
        # chunks of prompts, gpt-oss shapes, half the head rotated, in pairs; some rows are padding
        dict(name="norm_rope_append_8k", op="norm_rope_paged", T=8191, Hq=64, Hkv=8, d=64, rd=32, inter=True,
             norm=True, bs=64, pad=129),
        # the smallest call: two short sequences
        dict(name="varlen_tiny", op="varlen", Bc=1, cq_lo=5, cq_hi=5, cc_lo=700, cc_hi=700, Bd=1, dq_hi=1, dc_lo=40,
             dc_hi=40, Hq=8, Hkv=2, d=64, bs=16, window=0, n_sink=0, sinks=False),
        # 64 running requests, each with 1 to 8 drafted tokens to verify against 1K to 32K of context
        dict(name="varlen_verify_b64", op="varlen", Bc=0, cq_lo=0, cq_hi=0, cc_lo=0, cc_hi=0, Bd=64, dq_hi=8,
             dc_lo=1024, dc_hi=32768, Hq=32, Hkv=8, d=128, bs=16, window=0, n_sink=0, sinks=False),
        # one request of 131,072 tokens with 8 new ones
        dict(name="varlen_long_b1", op="varlen", Bc=0, cq_lo=0, cq_hi=0, cc_lo=0, cc_hi=0, Bd=1, dq_hi=-8,
             dc_lo=131072, dc_hi=131072, Hq=32, Hkv=8, d=128, bs=16, window=0, n_sink=0, sinks=False),
        # four prompt chunks beside 32 decoding requests, in one batch
        dict(name="varlen_mixed_b36", op="varlen", Bc=4, cq_lo=1024, cq_hi=2048, cc_lo=4096, cc_hi=16384, Bd=32,
             dq_hi=1, dc_lo=1024, dc_hi=32768, Hq=32, Hkv=8, d=128, bs=16, window=0, n_sink=0, sinks=False),
        # gpt-oss shapes: window 128, learned sinks, ragged chunks
        dict(name="varlen_gptoss_window", op="varlen", Bc=48, cq_lo=1, cq_hi=512, cc_lo=512, cc_hi=8192, Bd=16,
             dq_hi=1, dc_lo=1024, dc_hi=32768, Hq=64, Hkv=8, d=64, bs=16, window=128, n_sink=0, sinks=True),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["extend", "release", "norm_rope", "norm_rope_bwd", "norm_rope_paged", "varlen", "varlen",
                     "varlen"])
    bs = rng.choice([16, 32, 64, 128])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    rd = rng.choice([d, d, d // 2, 32, 48])
    if op == "extend":
        new_hi = _log(rng, 1, 255)
        return dict(op=op, B=_log(rng, 1, 512), len_lo=0, len_hi=_log(rng, 16, 8192), new_lo=rng.choice([0, 1]),
                    new_hi=new_hi, bs=bs, max_len=8192 + 256, pad=rng.choice([0, rng.randint(1, 999)]))
    if op == "release":
        return dict(op=op, B=_log(rng, 1, 512), len_lo=0, len_hi=_log(rng, 16, 8192), bs=bs, max_len=8192)
    if op in ("norm_rope", "norm_rope_bwd"):
        B = _log(rng, 1, 8)
        return dict(op=op, B=B, N=_log(rng, 1, 16384 // B), Hq=Hkv * min(group, 4), Hkv=Hkv, d=d, rd=rd,
                    inter=rng.random() < 0.4, norm=rng.random() < 0.8, pos=rng.random() < 0.5)
    if op == "norm_rope_paged":
        return dict(op=op, T=_log(rng, 1, 8192), Hq=Hkv * group, Hkv=Hkv, d=d, rd=rd, inter=rng.random() < 0.4,
                    norm=rng.random() < 0.8, bs=bs, pad=rng.choice([0, rng.randint(1, 99)]))
    window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    kind = rng.choice(["small", "decode", "chunk", "mixed"])
    c = dict(op=op, Bc=0, cq_lo=0, cq_hi=0, cc_lo=0, cc_hi=0, Bd=0, dq_hi=1, dc_lo=0, dc_hi=0, Hq=Hkv * group,
             Hkv=Hkv, d=d, bs=bs, window=window, n_sink=rng.choice([0, 4, 200]) if window else 0,
             sinks=rng.random() < 0.3)
    if kind in ("small", "decode", "mixed"):
        ctx = _log(rng, 16, 32768) if kind != "small" else _log(rng, 1, 512)
        c.update(Bd=_log(rng, 1, 40 if kind != "small" else 4), dq_hi=_log(rng, 1, 16), dc_lo=max(1, ctx // 4),
                 dc_hi=ctx)
    if kind in ("chunk", "mixed"):
        ctx = _log(rng, 64, 8192)
        q = _log(rng, 1, min(1024, ctx))
        c.update(Bc=_log(rng, 1, 4), cq_lo=max(1, q // 2), cq_hi=q, cc_lo=max(1, ctx // 2), cc_hi=ctx)
    return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _normal(shape, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(torch.bfloat16)


def _lengths(lo, hi, n, gen):
    return torch.randint(lo, hi + 1, (n,), generator=gen)


def _batch(case):
    """The sequences of a block-table case, in no order: lengths and new tokens. They go by the case alone (the
    inputs' shapes follow from them); the seed decides which sequence has which."""
    gen = torch.Generator().manual_seed(1)
    lens = _lengths(case["len_lo"], case["len_hi"], case["B"], gen)
    return lens, _lengths(case.get("new_lo", 0), case.get("new_hi", 0), case["B"], gen)


def _varlen_batch(case):
    """The same of a ragged batch, prompt chunks first: new tokens and context lengths."""
    gen = torch.Generator().manual_seed(1)
    cq = _lengths(case["cq_lo"], case["cq_hi"], case["Bc"], gen)
    cc = _lengths(case["cc_lo"], case["cc_hi"], case["Bc"], gen)
    # a negative dq_hi is the exact number of new tokens
    dq = _lengths(1, case["dq_hi"], case["Bd"], gen) if case["dq_hi"] > 0 else \
        torch.full((case["Bd"],), -case["dq_hi"], dtype=torch.int64)
    dc = _lengths(case["dc_lo"], case["dc_hi"], case["Bd"], gen)
    q = torch.cat([cq, dq])
    return q, torch.maximum(torch.cat([cc, dc]), q)


def _shuffled(pair, n, gen):
    at = torch.randperm(n, generator=gen)
    return [x[at] for x in pair]


def _layout(lens, bs, max_blocks, extra, gen, fill=-1):
    """A block table over a shuffled pool, the pool's size, and the block order: used blocks, then `extra` more."""
    need = (lens + bs - 1) // bs
    used = int(need.sum())
    perm = torch.randperm(used + extra, generator=gen).to(torch.int32)
    table = torch.full((len(lens), max_blocks), fill, dtype=torch.int32)
    j = torch.arange(max_blocks)[None, :]
    mask = j < need[:, None]
    table[mask] = perm[:used]
    return table, perm, used


def _rope_table(max_pos, rd, base=500000.0):
    """cos and sin [max_pos, rd / 2], the angles in 64 bits."""
    inv = base ** (-torch.arange(0, rd, 2, dtype=torch.float64) / rd)
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv[None, :]
    return ang.cos().float().cuda(), ang.sin().float().cuda()


def _weights(case, gen):
    if not case["norm"]:
        return None, None
    return [1.0 + 0.1 * torch.randn(case["d"], generator=gen, device="cuda") for _ in range(2)]


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    gpu = torch.Generator("cuda").manual_seed(seed)
    op, s = case["op"], dict(case)
    if op in ("extend", "release"):
        B, bs = case["B"], case["bs"]
        lens, new = _shuffled(_batch(case), B, cpu)
        extra = int(((lens + new + bs - 1) // bs - (lens + bs - 1) // bs).sum()) + 7
        table, perm, used = _layout(lens, bs, -(-case["max_len"] // bs), extra, cpu)
        free = torch.full((len(perm),), -1, dtype=torch.int32)
        free[:extra] = perm[used:]
        s.update(seq_lens=lens.int().cuda(), new_lens=new.int().cuda(), table=table.cuda(), free=free.cuda(),
                 num_free=torch.tensor([extra], dtype=torch.int32).cuda(), num_blocks=len(perm),
                 max_tokens=max(1, int(new.sum()) + case.get("pad", 0)),
                 finished=(torch.rand(B, generator=cpu) < 1 / 3).int().cuda())
        return s
    if op in ("norm_rope", "norm_rope_bwd"):
        B, N, Hq, Hkv, d = (case[k] for k in ("B", "N", "Hq", "Hkv", "d"))
        # one fused projection's output: q, k and v are views of it
        qkv = _normal((B, N, Hq + 2 * Hkv, d), gpu)
        s.update(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hkv], v=qkv[:, :, Hq + Hkv:])
        s["wq"], s["wk"] = _weights(case, gpu)
        s["cos"], s["sin"] = _rope_table(N, case["rd"])
        # packed documents: positions start again inside a row
        s["positions"] = (torch.arange(N, dtype=torch.int32) % max(1, N // 3 + 1)).repeat(B, 1).cuda() \
            if case["pos"] else None
        if op == "norm_rope_bwd":
            s.update(dq=_normal((B, Hq, N, d), gpu), dk=_normal((B, Hkv, N, d), gpu), dv=_normal((B, Hkv, N, d), gpu))
        return s
    if op == "norm_rope_paged":
        T, Hq, Hkv, d, bs = (case[k] for k in ("T", "Hq", "Hkv", "d", "bs"))
        max_pos = 32768
        qkv = _normal((T, Hq + 2 * Hkv, d), gpu)
        num_blocks = -(-T // bs) + 16
        slots = torch.randperm(num_blocks * bs, generator=cpu)[:T].int()
        pad = min(case["pad"], T - 1)
        if pad:
            slots[T - pad:] = -1
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], slots=slots.cuda(),
                 positions=_lengths(0, max_pos - 1, T, cpu).int().cuda(),
                 k_cache=_normal((num_blocks, bs, Hkv, d), gpu), v_cache=_normal((num_blocks, bs, Hkv, d), gpu))
        s["wq"], s["wk"] = _weights(case, gpu)
        s["cos"], s["sin"] = _rope_table(max_pos, case["rd"])
        return s
    # varlen: Bc chunks of prompts and Bd running requests, in any order
    Hq, Hkv, d, bs = (case[k] for k in ("Hq", "Hkv", "d", "bs"))
    q_len, ctx = _shuffled(_varlen_batch(case), case["Bc"] + case["Bd"], cpu)
    table, perm, used = _layout(ctx, bs, int((ctx.max() + bs - 1) // bs) + 1, 5, cpu)
    cu = torch.zeros(len(q_len) + 1, dtype=torch.int32)
    cu[1:] = q_len.cumsum(0)
    T = int(cu[-1])
    s.update(q=_normal((T, Hq, d), gpu), k_cache=_normal((len(perm), bs, Hkv, d), gpu),
             v_cache=_normal((len(perm), bs, Hkv, d), gpu), table=table.cuda(), cu=cu.cuda(),
             seq_lens=ctx.int().cuda(), max_seq_len=int(ctx.max()), spans=list(zip(q_len.tolist(), ctx.tolist())),
             sink_logits=torch.rand(Hq, generator=gpu, device="cuda") * 7 - 1 if case["sinks"] else None,
             out=torch.empty((T, Hq, d), dtype=torch.bfloat16, device="cuda"),
             lse=torch.empty((T, Hq), dtype=torch.float32, device="cuda"))
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _plain_extend(s):
    bs, L, n, free, table = s["bs"], s["seq_lens"].long(), s["new_lens"].long(), s["free"], s["table"]
    old, need = (L + bs - 1) // bs, (L + n + bs - 1) // bs
    off = (need - old).cumsum(0) - (need - old)
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    at = s["num_free"].long() - 1 - (off[:, None] + j - old[:, None])
    grown = (j >= old[:, None]) & (j < need[:, None])
    table.copy_(torch.where(grown, free[at.clamp(0, len(free) - 1)], table))
    cu = torch.cat([torch.zeros_like(n[:1]), n.cumsum(0)])
    t = torch.arange(s["max_tokens"], device=table.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=len(n) - 1)
    real = t < cu[-1]
    pos = torch.where(real, L[b] + t - cu[b], 0)
    slot = torch.where(real, table[b, pos // bs].long() * bs + pos % bs, -1)
    return {"seq_lens": (L + n).int(), "num_free": (s["num_free"] - (need - old).sum()).int(), "cu_q": cu.int(),
            "positions": pos.int(), "slots": slot.int(), "table": table}


def _plain_release(s):
    bs, L, free, table = s["bs"], s["seq_lens"].long(), s["free"], s["table"]
    have = (L + bs - 1) // bs * (s["finished"] != 0)
    off = have.cumsum(0) - have
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    to = s["num_free"].long() + off[:, None] + j
    # entries that stay go to one place behind the list
    to = torch.where(j < have[:, None], to, len(free))
    longer = torch.cat([free, free[:1]])
    longer[to] = table
    free.copy_(longer[:-1])
    return {"seq_lens": torch.where(s["finished"] != 0, 0, L).int(), "num_free": (s["num_free"] + have.sum()).int(),
            "free": free}


def _rotate(x, cos, sin, inter):
    """The first 2 * cos.shape[-1] elements of each head turned by the token's angles; x [..., H, d]."""
    h = cos.shape[-1]
    cos, sin = cos.unsqueeze(-2), sin.unsqueeze(-2)
    a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if inter else (x[..., :h], x[..., h:2 * h])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, w], -1).flatten(-2) if inter else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., 2 * h:]], -1)


def _angles(s):
    if s["positions"] is None:
        return s["cos"], s["sin"]
    at = s["positions"].long()
    return s["cos"][at], s["sin"][at]


_EPS = 1e-6


def _plain_norm_rope_one(x, w, cos, sin, inter):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * w
    return _rotate(x, cos, sin, inter)


def _plain_norm_rope(s):
    cos, sin = _angles(s)
    q = _plain_norm_rope_one(s["q"], s["wq"], cos, sin, s["inter"])
    k = _plain_norm_rope_one(s["k"], s["wk"], cos, sin, s["inter"])
    return [x.to(torch.bfloat16).transpose(1, 2).contiguous() for x in (q, k, s["v"])]


def _plain_norm_rope_bwd_one(x, w, dy, cos, sin, inter):
    """Gradients of one input and its weight; dy [B, H, N, d]."""
    dn = _rotate(dy.transpose(1, 2).float(), cos, -sin, inter)
    if w is None:
        return dn.to(torch.bfloat16), None
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS)
    n = x * r
    g = dn * w
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (dn * n).sum((0, 1, 2))


def _plain_norm_rope_bwd(s):
    cos, sin = _angles(s)
    dq, dwq = _plain_norm_rope_bwd_one(s["q"], s["wq"], s["dq"], cos, sin, s["inter"])
    dk, dwk = _plain_norm_rope_bwd_one(s["k"], s["wk"], s["dk"], cos, sin, s["inter"])
    return [dq, dk, s["dv"].transpose(1, 2).contiguous()] + ([dwq, dwk] if dwq is not None else [])


def _plain_norm_rope_paged(s):
    cos, sin = _angles(s)
    q = _plain_norm_rope_one(s["q"], s["wq"], cos, sin, s["inter"]).to(torch.bfloat16)
    k = _plain_norm_rope_one(s["k"], s["wk"], cos, sin, s["inter"]).to(torch.bfloat16)
    real = s["slots"] >= 0
    at = s["slots"][real].long()
    s["k_cache"].view(-1, *k.shape[1:])[at] = k[real]
    s["v_cache"].view(-1, *k.shape[1:])[at] = s["v"][real]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attend(q, k, v, n, window, n_sink, sinks):
    """q [n, Hq, d], k and v [ctx, Hkv, d] in one type: the newest n positions against the whole context."""
    ctx, Hkv, d = k.shape
    group = q.shape[1] // Hkv
    q = q.view(n, Hkv, group, d).permute(1, 2, 0, 3).reshape(Hkv, group * n, d)
    x = torch.matmul(q, k.permute(1, 2, 0)).view(Hkv, group, n, ctx) * (1 / math.sqrt(d))
    i = torch.arange(ctx - n, ctx, device=x.device)[:, None]
    j = torch.arange(ctx, device=x.device)[None, :]
    hidden = j > i
    if window:
        hidden |= (i - j >= window) & (j >= n_sink)
    x.masked_fill_(hidden, -math.inf)
    m = x.amax(-1, keepdim=True)
    if sinks is not None:
        m = torch.maximum(m, sinks.to(x.dtype).view(Hkv, group, 1, 1))
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    if sinks is not None:
        l = l + (sinks.to(x.dtype).view(Hkv, group, 1, 1) - m).exp()
    o = torch.matmul(p.view(Hkv, group * n, ctx), v.permute(1, 0, 2)).view(Hkv, group, n, d) / l
    lse = m + l.log()
    return o.permute(2, 0, 1, 3).reshape(n, Hkv * group, d), lse[..., 0].permute(2, 0, 1).reshape(n, Hkv * group)


def _plain_varlen(s):
    at = 0
    for b, (n, ctx) in enumerate(s["spans"]):  # sequences of any lengths: one after another
        blocks = s["table"][b, :-(-ctx // s["bs"])].long()
        k = s["k_cache"][blocks].flatten(0, 1)[:ctx].float()
        v = s["v_cache"][blocks].flatten(0, 1)[:ctx].float()
        o, lse = _attend(s["q"][at:at + n].float(), k, v, n, s["window"], s["n_sink"], s["sink_logits"])
        s["out"][at:at + n] = o
        s["lse"][at:at + n] = lse
        at += n
    return {"o": s["out"], "lse": s["lse"]}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _own(s):
    attn, op = _attn(), s["op"]
    if op == "extend":
        seq_lens, num_free, cu, pos, slots = attn.paged_extend(s["seq_lens"], s["new_lens"], s["table"], s["free"],
                                                               s["num_free"], s["bs"], s["num_blocks"],
                                                               s["max_tokens"])
        return {"seq_lens": seq_lens, "num_free": num_free, "cu_q": cu, "positions": pos, "slots": slots,
                "table": s["table"]}
    if op == "release":
        seq_lens, num_free = attn.paged_release(s["seq_lens"], s["finished"], s["table"], s["free"], s["num_free"],
                                                s["bs"], s["num_blocks"])
        return {"seq_lens": seq_lens, "num_free": num_free, "free": s["free"]}
    if op == "norm_rope":
        return list(attn.qk_norm_rope(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos"], s["sin"],
                                      positions=s["positions"], eps=_EPS, interleaved=s["inter"]))
    if op == "norm_rope_bwd":
        got = attn.qk_norm_rope_backward(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["dq"], s["dk"],
                                         s["dv"], positions=s["positions"], eps=_EPS, interleaved=s["inter"])
        return [g for g in got if g is not None]
    if op == "norm_rope_paged":
        q = attn.qk_norm_rope_paged(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos"], s["sin"], s["positions"],
                                    s["slots"], s["k_cache"], s["v_cache"], eps=_EPS, interleaved=s["inter"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    o, lse = attn.prefill_paged_varlen(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["seq_lens"],
                                       s["max_seq_len"], mask="window" if s["window"] else "causal",
                                       window=s["window"], n_sink=s["n_sink"], sinks=s["sink_logits"], out=s["out"],
                                       lse=s["lse"])
    return {"o": o, "lse": lse}


def run(state):
    if own:
        return _own(state)
    plain = {"extend": _plain_extend, "release": _plain_release, "norm_rope": _plain_norm_rope,
             "norm_rope_bwd": _plain_norm_rope_bwd, "norm_rope_paged": _plain_norm_rope_paged,
             "varlen": _plain_varlen}
    return plain[state["op"]](state)


# --------------------------------------------------------------------------
# work
# --------------------------------------------------------------------------
def _visible(n, ctx, window, n_sink):
    """(query, key) pairs seen, and keys that some query sees, of one sequence."""
    i = torch.arange(ctx - n, ctx, dtype=torch.int64)
    if not window:
        return int((i + 1).sum()), ctx
    near = torch.minimum(i + 1, torch.tensor(window))
    first = (i - near + 1)
    pairs = int((near + torch.minimum(first, torch.tensor(n_sink))).sum())
    lo = int(first[0])
    return pairs, ctx - lo + min(lo, n_sink)


def work(case):
    op = case["op"]
    if op in ("extend", "release"):
        B, bs = case["B"], case["bs"]
        lens, new = _batch(case)
        have = (lens + bs - 1) // bs
        if op == "release":  # lengths and flags in, lengths out; the freed entries from the table to the list
            return {"bytes": 12 * B + 8 * int(have.sum()) / 3, "flops": 0}
        grown = int(((lens + new + bs - 1) // bs - have).sum())
        # lengths in and out, cu, the entry that each sequence goes on in; new entries from the list to the table;
        # a position and a slot for each token
        return {"bytes": 20 * B + 8 * grown + 8 * (int(new.sum()) + case["pad"]), "flops": 0}
    if op in ("norm_rope", "norm_rope_bwd", "norm_rope_paged"):
        T = case["T"] if op == "norm_rope_paged" else case["B"] * case["N"]
        Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
        angles = min(T, case.get("N", T)) * case["rd"] * 4
        if op == "norm_rope_bwd":  # x of q and k (none without norms), three gradients in, three out
            x = (Hq + Hkv) * d * 2 if case["norm"] else 0
            return {"bytes": T * (x + 4 * (Hq + 2 * Hkv) * d) + angles, "flops": 20 * T * (Hq + Hkv) * d}
        return {"bytes": T * 4 * (Hq + 2 * Hkv) * d + angles, "flops": 8 * T * (Hq + Hkv) * d}
    q_len, ctx = _varlen_batch(case)
    seen = [_visible(n, c, case["window"], case["n_sink"]) for n, c in zip(q_len.tolist(), ctx.tolist())]
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    return {"bytes": sum(k for _, k in seen) * Hkv * d * 4 + int(q_len.sum()) * Hq * (d * 4 + 4),
            "flops": 4 * d * Hq * sum(p for p, _ in seen)}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_norm_rope_one(x, w, s):
    """One head row after another as complex numbers: the rotation is a product with exp(i angle)."""
    n = x
    if w is not None:
        n = x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + _EPS).sqrt() * w
    pos = s["positions"].long() if s["positions"] is not None else torch.arange(x.shape[1], device=x.device)
    turn = torch.complex(s["cos"].double()[pos], s["sin"].double()[pos]).unsqueeze(-2)
    h = turn.shape[-1]
    if s["inter"]:
        z = torch.view_as_complex(n[..., :2 * h].unflatten(-1, (h, 2)).contiguous()) * turn
        y = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(n[..., :h].contiguous(), n[..., h:2 * h].contiguous()) * turn
        y = torch.cat([z.real, z.imag], -1)
    return torch.cat([y, n[..., 2 * h:]], -1)


def exact(case, seed):
    op = case["op"]
    if op in ("extend", "release"):
        return None
    s = prepare(case, seed)
    if op == "varlen":
        return _exact_varlen(s)
    x = [s["q"].double().requires_grad_(), s["k"].double().requires_grad_()]
    w = [None if v is None else v.double().requires_grad_() for v in (s["wq"], s["wk"])]
    y = [_exact_norm_rope_one(a, b, s) for a, b in zip(x, w)]
    if op == "norm_rope":
        return [t.detach().transpose(1, 2).contiguous() for t in y + [s["v"].double()]]
    if op == "norm_rope_bwd":
        leaves = x + [v for v in w if v is not None]
        dy = [s["dq"].double().transpose(1, 2), s["dk"].double().transpose(1, 2)]
        g = torch.autograd.grad(y, leaves, dy)
        return [g[0], g[1], s["dv"].double().transpose(1, 2).contiguous(), *g[2:]]
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    real = s["slots"] >= 0
    blk, off = (s["slots"][real] // s["bs"]).long(), (s["slots"][real] % s["bs"]).long()
    k_cache[blk, off] = y[1].detach()[real]
    v_cache[blk, off] = s["v"].double()[real]
    return {"q": y[0].detach(), "k_cache": k_cache, "v_cache": v_cache}


def _exact_varlen(s):
    """Head by head: scores, the visible ones' softmax with the sink's weight in its sum, the mean of V."""
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    group = s["Hq"] // s["Hkv"]
    at = 0
    for b, (n, ctx) in enumerate(s["spans"]):
        token = torch.arange(ctx, device="cuda")
        slot = s["table"][b].long()[token // s["bs"]], token % s["bs"]
        back = torch.arange(ctx - n, ctx, device="cuda")[:, None] - token[None, :]
        seen = back >= 0
        if s["window"]:
            seen = seen & ((back < s["window"]) | (token[None, :] < s["n_sink"]))
        for kv in range(s["Hkv"]):
            k, v = s["k_cache"][slot][:, kv].double(), s["v_cache"][slot][:, kv].double()
            for h in range(kv * group, (kv + 1) * group):
                x = s["q"][at:at + n, h].double() @ k.T / math.sqrt(s["d"])
                x = torch.where(seen, x, -math.inf)
                if s["sink_logits"] is not None:
                    x = torch.cat([x, s["sink_logits"][h].double().expand(n, 1)], 1)
                total = torch.logsumexp(x, 1)
                o[at:at + n, h] = (x[:, :ctx] - total[:, None]).exp() @ v
                lse[at:at + n, h] = total
        at += n
    return {"o": o, "lse": lse}
