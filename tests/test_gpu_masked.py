"""dit_attn_fwd_masked against the fp64 definition: every mask and score change, shared heads, one
query to many, rows that see nothing, and what lies under the masks."""

import numpy as np
import pytest

from gpu_util import assert_bf16_parity, metrics
from oracle import block

pytestmark = pytest.mark.gpu


def _np(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def _bf16(shape, seed, scale=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _i32(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _qkv(B, H, Hk, S_q, S_kv, D, seed=0, loud=1.0):
    return _bf16((B, H, S_q, D), seed, loud), _bf16((B, Hk, S_kv, D), seed + 1), _bf16((B, Hk, S_kv, D), seed + 2)


def _check(lsa, q, k, v, **kw):
    """Runs the call, compares with the definition, returns (out, lse)."""
    scale = kw.pop("scale", q.shape[-1] ** -0.5)
    o, l = lsa.masked_attention(q, k, v, scale=scale, **kw)
    host = {n: (x.cpu().numpy() if hasattr(x, "cpu") else x) for n, x in kw.items()}
    ro, rl = block.masked_attention(_np(q), _np(k), _np(v), scale, **host)
    m = metrics(_np(o), ro, _np(l), rl)
    assert_bf16_parity(m, str({n: x for n, x in kw.items() if not hasattr(x, "cpu")}))
    empty = np.isneginf(rl)
    assert np.all(_np(o)[empty] == 0)
    assert lsa.dit_device_status() == 0
    return o, l


LENGTHS = [(1, 1), (1, 5), (7, 7), (77, 77), (128, 128), (129, 257), (200, 130), (300, 300), (64, 700), (513, 513)]


@pytest.mark.parametrize("S_q,S_kv", LENGTHS)
@pytest.mark.parametrize("D", [64, 128])
def test_lengths_and_causal(cuda_lib, S_q, S_kv, D):
    q, k, v = _qkv(2, 4, 2, S_q, S_kv, D, S_q)
    _check(cuda_lib, q, k, v)
    _check(cuda_lib, q, k, v, causal=True)           # S_q > S_kv: the first queries see nothing


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (6, 1), (8, 2)])
def test_everything_at_once(cuda_lib, D, H, Hk):
    import torch
    S = 333
    q, k, v = _qkv(2, H, Hk, S, S, D, 3, 3.0)
    doc = np.repeat(np.arange(9), 37).reshape(1, -1).repeat(2, 0)
    doc[0, 300:] = -1
    doc[1, :41] = -7
    slopes = torch.tensor([0.02 * 2.0 ** h for h in range(H)], device="cuda")
    kw = dict(softcap=4.0, slopes=slopes, causal=True, prefix=_i32([150, 20]), q_doc=_i32(doc), kv_doc=_i32(doc))
    for drop in ((), ("softcap",), ("slopes",), ("causal", "prefix"), ("prefix",), ("q_doc", "kv_doc")):
        _check(cuda_lib, q, k, v, **{n: x for n, x in kw.items() if n not in drop})


def test_prefix_and_starts(cuda_lib):
    S_q, S_kv = 150, 400
    q, k, v = _qkv(4, 2, 1, S_q, S_kv, 64, 5)
    for start in ([0, 100, 250, 399], [-30, -200, 500, 250]):
        for prefix in (None, [0, 1, 129, 400], [1000, -3, 128, 256]):
            _check(cuda_lib, q, k, v, causal=True, q_start=_i32(start), prefix=None if prefix is None else _i32(prefix))


def test_documents_in_any_order(cuda_lib):
    r = np.random.default_rng(0)
    q, k, v = _qkv(2, 2, 2, 260, 515, 128, 7)
    qd, kd = r.integers(-1, 4, (2, 260)), r.integers(-1, 3, (2, 515))      # document 3 has no key
    _check(cuda_lib, q, k, v, q_doc=_i32(qd), kv_doc=_i32(kd))
    qd[0], kd[0] = 2 ** 31 - 1, 2 ** 31 - 1
    kd[1] = -2 ** 31                                                         # a sequence of padding only
    _check(cuda_lib, q, k, v, q_doc=_i32(qd), kv_doc=_i32(kd))


@pytest.mark.parametrize("cap", [0.5, 5.0, 50.0])
def test_caps(cuda_lib, cap):
    for loud, D in ((1.0, 64), (8.0, 128)):
        q, k, v = _qkv(1, 2, 1, 200, 300, D, 9, loud)
        _check(cuda_lib, q, k, v, softcap=cap)
        _check(cuda_lib, q, k, v, softcap=cap, causal=True)


def test_bias_both_sides_and_negative_slopes(cuda_lib):
    import torch
    q, k, v = _qkv(1, 4, 4, 300, 300, 64, 11)
    slopes = torch.tensor([1.0, 0.01, 0.0, -0.05], device="cuda")
    _check(cuda_lib, q, k, v, slopes=slopes)
    _check(cuda_lib, q, k, v, slopes=slopes, causal=True, prefix=_i32([170]))


@pytest.mark.parametrize("B,H,Hk,S_q,S_kv,D", [(1, 1, 1, 1, 5000, 64), (3, 8, 2, 1, 4097, 128), (2, 24, 24, 1, 1000, 64),
                                               (1, 16, 1, 5, 9001, 128), (1, 40, 8, 3, 2100, 128), (2, 5, 5, 40, 3000, 64)])
def test_few_queries_against_a_cache(cuda_lib, B, H, Hk, S_q, S_kv, D):
    import torch
    q, k, v = _qkv(B, H, Hk, S_q, S_kv, D, 13)
    _check(cuda_lib, q, k, v, causal=True)
    start = _i32([0, S_kv - S_q, S_kv // 3][:B])
    _check(cuda_lib, q, k, v, causal=True, q_start=start, slopes=torch.full((H,), 0.003, device="cuda"))
    _check(cuda_lib, q, k, v, softcap=9.0)
    kd = np.zeros((B, S_kv), int)
    kd[:, S_kv // 2:] = -1
    _check(cuda_lib, q, k, v, q_doc=_i32(np.zeros((B, S_q), int)), kv_doc=_i32(kd))


def test_no_keys_no_queries(cuda_lib):
    import torch
    q, k, v = _qkv(2, 2, 1, 5, 9, 64)
    o, l = cuda_lib.masked_attention(q, k[:, :, :0].contiguous(), v[:, :, :0].contiguous())
    assert torch.all(o == 0) and torch.all(torch.isneginf(l))
    o, l = cuda_lib.masked_attention(q[:, :, :0].contiguous(), k, v, causal=True)
    assert o.shape == (2, 2, 0, 64) and l.shape == (2, 2, 0)
    o, l = cuda_lib.masked_attention(q, k, v, causal=True, q_start=_i32([-9, -100]))
    assert torch.all(o == 0) and torch.all(torch.isneginf(l))
    o, l = cuda_lib.masked_attention(q, k, v, with_lse=False)
    assert l is None


@pytest.mark.parametrize("S_q", [1, 6, 300])
@pytest.mark.parametrize("D", [64, 128])
def test_what_lies_under_the_masks_does_not_matter(cuda_lib, S_q, D):
    import torch
    S_kv = 700
    q, k, v = _qkv(2, 4, 2, S_q, S_kv, D, 17)
    start = [300 - min(S_q, 300), 650 - S_q]
    kd = np.zeros((2, S_kv), int)
    kd[:, 40:55] = 1                                 # another document, inside a tile
    kd[1, 5] = -1
    kw = dict(causal=True, q_start=_i32(start), q_doc=_i32(np.zeros((2, S_q), int)), kv_doc=_i32(kd))
    want = cuda_lib.masked_attention(q, k, v, **kw)
    hidden = kd != 0
    for b in range(2):
        hidden[b, start[b] + S_q:] = True
    for bad in (float("nan"), float("inf"), -float("inf"), 3.0e38):
        kb, vb = k.clone(), v.clone()
        for b in range(2):
            m = torch.from_numpy(hidden[b]).cuda()
            kb[b, :, m] = bad
            vb[b, :, m] = bad
        got = cuda_lib.masked_attention(q, kb, vb, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), bad


@pytest.mark.parametrize("S_q", [1, 300])
def test_a_bad_value_stays_with_the_queries_that_see_it(cuda_lib, S_q):
    """Packed documents: NaN and infinities in one leave the others alone, inside the same tiles too."""
    import torch
    S = 300
    q, k, v = _qkv(1, 2, 1, S_q, S, 64, 19)
    kd = np.repeat(np.arange(6), 50)[None]
    qd = kd if S_q == S else np.array([[2]])
    want = cuda_lib.masked_attention(q, k, v, q_doc=_i32(qd), kv_doc=_i32(kd))
    v[0, 0, 60, 3], v[0, 0, 260, 5], k[0, 0, 270, 1] = float("nan"), float("inf"), float("nan")
    got = cuda_lib.masked_attention(q, k, v, q_doc=_i32(qd), kv_doc=_i32(kd))
    good = torch.from_numpy((qd[0] != 1) & (qd[0] != 5)).cuda()
    assert torch.equal(got[0][:, :, good], want[0][:, :, good]) and torch.equal(got[1][:, :, good], want[1][:, :, good])
    if S_q == S:
        assert torch.all(torch.isnan(got[0][0, :, 50:100, 3])) and not torch.any(torch.isfinite(got[0][0, :, 250:, 5]))


def test_large_scores(cuda_lib):
    """Scores of hundreds, rising along the keys: every tile moves the running maximum."""
    q, k, v = _qkv(1, 2, 1, 150, 640, 64, 21)
    import torch
    k = (k.float() * torch.linspace(0.1, 12.0, 640, device="cuda")[None, None, :, None]).to(torch.bfloat16)
    o, l = cuda_lib.masked_attention(q, k, v, scale=0.5, causal=True)
    ro, rl = block.masked_attention(_np(q), _np(k), _np(v), 0.5, causal=True)
    m = metrics(_np(o), ro, _np(l), rl)
    assert_bf16_parity(m)


def test_same_results_again_other_streams_and_graphs(cuda_lib):
    import torch
    for S_q, S_kv in ((300, 300), (1, 3000)):
        q, k, v = _qkv(2, 8, 2, S_q, S_kv, 128, 23)
        doc = _i32(np.zeros((2, S_kv), int))
        qd = _i32(np.zeros((2, S_q), int))
        call = lambda **kw: cuda_lib.masked_attention(q, k, v, causal=True, q_doc=qd, kv_doc=doc, **kw)
        want = call()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(3)]
        got = [call(stream=s) for s in streams for _ in range(3)]     # calls side by side
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g in got for a, b in zip(want, g))
        g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g1):
            c1 = call()
        with torch.cuda.graph(g2):
            c2 = call()
        q.neg_()
        doc[:, ::3] = -1
        g1.replay()
        g2.replay()
        now = call()
        assert all(torch.equal(a, b) for a, b in zip(now, c1)) and all(torch.equal(a, b) for a, b in zip(now, c2))
    assert cuda_lib.dit_device_status() == 0
