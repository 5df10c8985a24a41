"""CPU checks of the C ABI's refusals for the operators around the paged cache:
every call here fails validation, so nothing is launched."""

import ctypes

import pytest

from exact_softmax_attention_causal_b200 import _lib

FAKE = ctypes.c_void_p(0x10000)  # aligned, never dereferenced
ODD = ctypes.c_void_p(0x10002)
NULL = ctypes.c_void_p(0)
INVALID, UNSUPPORTED, WORKSPACE = _lib.ATTN_ERR_INVALID_ARG, _lib.ATTN_ERR_UNSUPPORTED, _lib.ATTN_ERR_WORKSPACE


def _extend(**kw):
    a = dict(sl=FAKE, nl=FAKE, bt=FAKE, fb=FAKE, nf=FAKE, slo=FAKE, nfo=FAKE, cu=FAKE, pos=FAKE, slots=FAKE, B=2, nb=10,
             bs=16, mb=4, cap=10, mt=5)
    a.update(kw)
    return _lib.lib().attn_paged_extend(*a.values(), NULL, NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(sl=NULL), INVALID), (dict(nl=NULL), INVALID), (dict(bt=NULL), INVALID), (dict(fb=NULL), INVALID),
    (dict(nf=NULL), INVALID), (dict(slo=NULL), INVALID), (dict(nfo=NULL), INVALID), (dict(cu=NULL), INVALID),
    (dict(pos=NULL), INVALID), (dict(slots=NULL), INVALID), (dict(bt=ODD), INVALID), (dict(slots=ODD), INVALID),
    (dict(B=0), INVALID), (dict(nb=0), INVALID), (dict(bs=0), INVALID), (dict(mb=-1), INVALID), (dict(cap=0), INVALID),
    (dict(mt=-1), INVALID), (dict(B=8193), UNSUPPORTED), (dict(nb=1 << 27), UNSUPPORTED), (dict(mb=1 << 27), UNSUPPORTED),
    (dict(B=8192, mb=1 << 18, bs=1), UNSUPPORTED),
])
def test_extend_rejects_bad_arguments(kw, code):
    assert _extend(**kw) == code


def _release(**kw):
    a = dict(sl=FAKE, fin=FAKE, bt=FAKE, fb=FAKE, nf=FAKE, slo=FAKE, nfo=FAKE, B=2, nb=10, bs=16, mb=4, cap=10)
    a.update(kw)
    return _lib.lib().attn_paged_release(*a.values(), NULL, NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(sl=NULL), INVALID), (dict(fin=NULL), INVALID), (dict(fb=NULL), INVALID), (dict(nfo=NULL), INVALID),
    (dict(fin=ODD), INVALID), (dict(B=0), INVALID), (dict(bs=-4), INVALID), (dict(B=8193), UNSUPPORTED),
    (dict(mb=1 << 27), UNSUPPORTED),
])
def test_release_rejects_bad_arguments(kw, code):
    assert _release(**kw) == code


def _strides(n, bad=None):
    s = (ctypes.c_int64 * n)(*[128] * n)
    if bad is not None:
        s[bad] = 100
    return s


NORM_ROPE = [
    (dict(q=NULL), INVALID), (dict(k=NULL), INVALID), (dict(wq=NULL), INVALID), (dict(cos=NULL), INVALID),
    (dict(sin=NULL), INVALID), (dict(q=ctypes.c_void_p(0x10008)), INVALID), (dict(wk=ctypes.c_void_p(0x10004)), INVALID),
    (dict(pos=ODD), INVALID), (dict(Hq=0), INVALID), (dict(N=0), INVALID), (dict(rd=0), INVALID), (dict(rd=144), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("inf")), INVALID), (dict(max_pos=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(d=256), UNSUPPORTED), (dict(rd=24), UNSUPPORTED), (dict(Hq=70000), UNSUPPORTED),
]


def _norm_rope(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, st=_strides(9), wq=FAKE, wk=FAKE, bf=0, cos=FAKE, sin=FAKE, pos=NULL, qo=FAKE, ko=FAKE,
             vo=FAKE, B=1, N=8, Hq=4, Hkv=2, d=128, rd=128, max_pos=64, eps=1e-6, inter=0)
    a.update(kw)
    return _lib.lib().attn_qk_norm_rope(*a.values(), NULL, NULL)


@pytest.mark.parametrize("kw,code", NORM_ROPE + [
    (dict(v=NULL), INVALID), (dict(qo=NULL), INVALID), (dict(vo=ctypes.c_void_p(0x10008)), INVALID), (dict(st=None), INVALID),
    (dict(st=_strides(9, 8)), INVALID), (dict(B=0), INVALID), (dict(max_pos=7), INVALID), (dict(B=1 << 30), UNSUPPORTED),
])
def test_norm_rope_rejects_bad_arguments(kw, code):
    assert _norm_rope(**kw) == code


def _norm_rope_paged(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, st=_strides(6), wq=FAKE, wk=FAKE, bf=0, cos=FAKE, sin=FAKE, pos=FAKE, slots=FAKE, qo=FAKE,
             kc=FAKE, vc=FAKE, N=8, Hq=4, Hkv=2, d=128, nb=4, bs=16, rd=128, max_pos=64, eps=1e-6, inter=0)
    a.update(kw)
    return _lib.lib().attn_qk_norm_rope_paged(*a.values(), NULL, NULL)


@pytest.mark.parametrize("kw,code", NORM_ROPE + [
    (dict(v=NULL), INVALID), (dict(slots=NULL), INVALID), (dict(pos=NULL), INVALID), (dict(kc=NULL), INVALID),
    (dict(slots=ODD), INVALID), (dict(nb=0), INVALID), (dict(bs=0), INVALID), (dict(st=_strides(6, 1)), INVALID),
])
def test_norm_rope_paged_rejects_bad_arguments(kw, code):
    assert _norm_rope_paged(**kw) == code


def _norm_rope_bwd(**kw):
    a = dict(q=FAKE, k=FAKE, st=_strides(6), wq=FAKE, wk=FAKE, bf=0, cos=FAKE, sin=FAKE, pos=NULL, dzq=FAKE, dzk=FAKE, dzv=FAKE,
             dq=FAKE, dk=FAKE, dv=FAKE, gst=_strides(9), dwq=FAKE, dwk=FAKE, B=1, N=8, Hq=4, Hkv=2, d=128, rd=128, max_pos=64,
             eps=1e-6, inter=0, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return _lib.lib().attn_qk_norm_rope_backward(*a.values(), NULL, NULL)


@pytest.mark.parametrize("kw,code", NORM_ROPE + [
    (dict(dzv=NULL), INVALID), (dict(dq=NULL), INVALID), (dict(dwq=NULL), INVALID), (dict(dv=ctypes.c_void_p(0x10008)), INVALID),
    (dict(gst=None), INVALID), (dict(gst=_strides(9, 7)), INVALID),
])
def test_norm_rope_backward_rejects_bad_arguments(kw, code):
    assert _norm_rope_bwd(**kw) == code


def test_norm_rope_backward_workspace_rejects_bad_sizes():
    f = _lib.lib().attn_qk_norm_rope_backward_workspace_bytes
    assert f(0, 8, 4, 2, 128) == 0 and f(1, 8, 4, 2, 96) == 0


def _varlen(**kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, cu=FAKE, sl=FAKE, sinks=NULL, o=FAKE, lse=NULL, B=2, T=10, Hq=8, Hkv=2, d=128,
             nb=10, bs=16, mb=8, msl=128, mask=1, window=0, n_sink=0, scale=0.1, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return _lib.lib().attn_prefill_paged_varlen(*a.values(), NULL, NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(q=NULL), INVALID), (dict(vc=NULL), INVALID), (dict(bt=NULL), INVALID), (dict(cu=NULL), INVALID),
    (dict(sl=NULL), INVALID), (dict(o=NULL), INVALID), (dict(q=ctypes.c_void_p(0x10008)), INVALID), (dict(cu=ODD), INVALID),
    (dict(sinks=ODD), INVALID), (dict(lse=ODD), INVALID), (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(nb=0), INVALID),
    (dict(Hq=6, Hkv=4), INVALID), (dict(mb=7), INVALID), (dict(msl=0), INVALID), (dict(mask=7), INVALID),
    (dict(mask=2, window=0), INVALID), (dict(n_sink=1), INVALID), (dict(mask=2, window=4, n_sink=-1), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(bs=8, mb=16), UNSUPPORTED), (dict(bs=48, mb=3), UNSUPPORTED),
    (dict(T=1 << 28), UNSUPPORTED), (dict(mb=1 << 27, msl=(1 << 30) + 1), UNSUPPORTED),
])
def test_varlen_rejects_bad_arguments(kw, code):
    assert _varlen(**kw) == code


def test_varlen_workspace_rejects_bad_head_dimensions():
    assert _lib.lib().attn_prefill_paged_varlen_workspace_bytes(96) == 0
