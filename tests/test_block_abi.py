"""Refusals of the norm, rotary and masked-attention calls: host-side validation, no GPU needed.
Every call here has an invalid argument (or nothing to do), so nothing is ever launched."""

import ctypes

import pytest

A = 1 << 40
G = 1 << 30                      # distance between the fake buffers


@pytest.fixture(scope="module")
def lsa():
    import __graft_entry__
    __graft_entry__.build()
    import long_sequence_attention_b200 as lsa
    return lsa


def _norm(lsa, **kw):
    a = dict(x=A, ld=64, r=A + G, w=A + 2 * G, out=A + 3 * G, so=A + 4 * G, ds=None, rows=4, C=64, eps=1e-6, dt=0, od=0,
             group=0)
    a.update(kw)
    return lsa.lib.dit_rms_norm(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(out=None), 1), (dict(rows=-1), 1), (dict(C=0), 1), (dict(ld=63), 1), (dict(dt=1), 1),
    (dict(od=3), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(group=128), 1), (dict(od=1), 1), (dict(od=1, ds=A + 5 * G, group=64), 1), (dict(ds=A + 5 * G), 1),
    (dict(r=None), 1),                                         # a stream without a residual
    (dict(x=A + 1), 3), (dict(dt=2, x=A + 2), 3), (dict(od=1, ds=A + 5 * G + 2), 3), (dict(od=2, out=A + 3 * G + 2), 3),
    (dict(out=A + 64), 1), (dict(out=A + G), 1), (dict(out=A + 2 * G), 1), (dict(out=A + 4 * G + 16), 1),
    (dict(so=A + 2), 1), (dict(ld=65, so=A), 1), (dict(so=A + G + 64), 1), (dict(so=A + 2 * G), 1),
    (dict(od=1, ds=A + 3 * G), 1), (dict(rows=1 << 40), 1),
    (dict(rows=0, x=None), 0),
])
def test_norm(lsa, kw, code):
    assert _norm(lsa, **kw) == code


def _rope(lsa, **kw):
    a = dict(q=A, k=A + G, qs=(8192, 256, 128), ks=(8192, 256, 128), wq=None, wk=None, eps=1e-6, pos=A + 2 * G, psb=0,
             freqs=A + 3 * G, per=(64,), axes=1, rot=128, inter=0, mag=1.0, qo=A + 4 * G, ko=A + 5 * G, dq=None, dk=None,
             B=2, S=32, H=2, Hk=2, D=128, od=0)
    a.update(kw)
    for n in ("qs", "ks"):
        a[n] = None if a[n] is None else (ctypes.c_longlong * 3)(*a[n])
    a["per"] = None if a["per"] is None else (ctypes.c_int * 3)(*a["per"])
    return lsa.lib.dit_rope_qk(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(pos=None), 1), (dict(freqs=None), 1), (dict(qo=None), 1),
    (dict(ko=None), 1), (dict(qs=None), 1), (dict(ks=None), 1), (dict(per=None), 1), (dict(B=-1), 1), (dict(S=-1), 1),
    (dict(H=0), 1), (dict(Hk=-1), 1), (dict(Hk=0), 1), (dict(D=96), 2), (dict(D=256), 2), (dict(rot=130, per=(65,)), 1),
    (dict(rot=0, per=(0,)), 1), (dict(rot=127), 1), (dict(rot=24, per=(12,)), 2), (dict(per=(63,)), 1),
    (dict(axes=0), 1), (dict(axes=4), 1), (dict(axes=2, per=(65, -1)), 1), (dict(axes=2, per=(32, 33)), 1),
    (dict(eps=-1.0), 1), (dict(mag=float("nan")), 1), (dict(od=2), 1), (dict(od=1), 1), (dict(dq=A + 6 * G), 1),
    (dict(od=1, dq=A + 6 * G), 1), (dict(psb=31), 1), (dict(qs=(8192, 256, 4)), 3), (dict(qs=(8192, -256, 128)), 1),
    (dict(q=A + 8), 3), (dict(k=A + G + 2), 3), (dict(qo=A + 4 * G + 8), 3), (dict(pos=A + 2 * G + 2), 3),
    (dict(freqs=A + 3 * G + 4), 3), (dict(wq=A + 6 * G + 2), 3),
    (dict(qo=A), 1), (dict(qo=A + G), 1), (dict(ko=A + 4 * G), 1), (dict(qo=A + 2 * G), 1), (dict(ko=A + 3 * G), 1),
    (dict(B=0, q=None), 0), (dict(S=0), 0),
])
def test_rope(lsa, kw, code):
    assert _rope(lsa, **kw) == code


def _attn(lsa, **kw):
    a = dict(q=A, k=A + G, v=A + 2 * G, out=A + 3 * G, lse=A + 4 * G, B=2, H=4, Hk=2, S_q=32, S_kv=48, D=64, scale=0.1,
             cap=0.0, slopes=None, causal=1, start=None, prefix=None, qd=None, kd=None, ws=A + 8 * G, wsn=1 << 28)
    a.update(kw)
    return lsa.lib.dit_attn_fwd_masked(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(out=None), 1), (dict(B=-1), 1), (dict(H=0), 1),
    (dict(Hk=0), 1), (dict(Hk=3), 1), (dict(S_q=-1), 1), (dict(S_kv=-1), 1), (dict(S_kv=(1 << 30) + 1), 1),
    (dict(D=96), 2), (dict(scale=0.0), 1), (dict(scale=float("inf")), 1), (dict(cap=-1.0), 1),
    (dict(cap=float("nan")), 1), (dict(cap=float("inf")), 1), (dict(qd=A + 5 * G), 1), (dict(kd=A + 5 * G), 1),
    (dict(causal=0, prefix=A + 5 * G), 1), (dict(q=A + 8), 3), (dict(v=A + 2 * G + 2), 3), (dict(lse=A + 4 * G + 1), 3),
    (dict(slopes=A + 5 * G + 2), 3), (dict(start=A + 5 * G + 2), 3), (dict(ws=A + 8 * G + 8), 3),
    (dict(out=A), 1), (dict(out=A + 2 * G), 1), (dict(lse=A + 3 * G), 1), (dict(lse=A + G), 1),
    (dict(slopes=A + 3 * G + 16), 1), (dict(qd=A + 4 * G, kd=A + 5 * G), 1),
    (dict(B=0, q=None), 0), (dict(S_q=0), 0),
])
def test_masked(lsa, kw, code):
    assert _attn(lsa, **kw) == code


def test_python_checks(lsa):
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        lsa.rms_norm(x)                                        # not a CUDA tensor
    with pytest.raises(ValueError):
        lsa.rope_qk(x.view(1, 1, 4, 64), None, None, None)
    with pytest.raises(ValueError):
        lsa.masked_attention(x.view(1, 1, 4, 64), x.view(1, 1, 4, 64), x.view(1, 1, 4, 64))
    for kw in (dict(rot=7), dict(rot=8, axis_pairs=[1, 2]), dict(rot=8, scaling="other"), dict(rot=8, theta=0.0),
               dict(rot=8, factor=0.5), dict(rot=8, scaling="by_parts", factor=2.0)):
        with pytest.raises(ValueError):
            lsa.rope_frequencies(**kw)
