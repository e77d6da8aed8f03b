"""dit_attn_fwd_masked on long and mixed calls, against the definition in fp64 on the GPU (plain matrix products, row
blocks at a time): walks of more than 32 tiles, more units than CTAs, every mask together, random calls."""

import math
import random

import pytest

from gpu_util import BF16_MAX_ABS, BF16_REL_L2, LSE_MAX_ABS

pytestmark = pytest.mark.gpu


def _reference(q, k, v, scale, softcap=0.0, slopes=None, causal=False, q_start=None, prefix=None, q_doc=None, kv_doc=None):
    import torch
    B, H, S_q, D = q.shape
    H_kv, S_kv = k.shape[1], k.shape[2]
    out = torch.zeros(B, H, S_q, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, S_q), -math.inf, dtype=torch.float64, device="cuda")
    key = torch.arange(S_kv, device="cuda")
    for b in range(B):
        start = S_kv - S_q if q_start is None else int(q_start[b])
        for r in range(0, S_q, 2048):
            pos = start + torch.arange(r, min(r + 2048, S_q), device="cuda")[:, None]
            hide = torch.zeros(pos.shape[0], S_kv, dtype=torch.bool, device="cuda")
            if causal:
                hide |= (key > pos) & (key >= (0 if prefix is None else int(prefix[b])))
            if q_doc is not None:
                mine = q_doc[b, r:r + 2048, None]
                hide |= (mine != kv_doc[b]) | (mine < 0)
            for h in range(H):
                s = q[b, h, r:r + 2048].double() @ k[b, h * H_kv // H].double().T * scale
                if softcap:
                    s = softcap * torch.tanh(s / softcap)
                if slopes is not None:
                    s = s - slopes[h].double() * (pos - key).abs()
                s = s.masked_fill(hide, -math.inf)
                l = torch.logsumexp(s, 1)
                lse[b, h, r:r + 2048] = l
                p = torch.exp(s - l[:, None]).masked_fill(hide, 0.0)
                out[b, h, r:r + 2048] = p @ v[b, h * H_kv // H].double()
    return out, lse


def _check(lsa, q, k, v, **kw):
    import torch
    scale = q.shape[-1] ** -0.5
    o, l = lsa.masked_attention(q, k, v, scale=scale, **kw)
    ro, rl = _reference(q, k, v, scale, **kw)
    o, l = o.double(), l.double()
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(l), empty) and torch.all(o[empty] == 0) and not torch.any(torch.isnan(o))
    if not torch.all(empty):
        assert (l - rl)[~empty].abs().max() <= LSE_MAX_ABS
        assert (o - ro).norm() <= BF16_REL_L2 * ro.norm() and (o - ro).abs().max() <= BF16_MAX_ABS
    assert lsa.dit_device_status() == 0


def _rand(shape, g, scale=1.0):
    import torch
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _docs(rng, B, S, shuffled=False):
    import torch
    ids = []
    for _ in range(B):
        row = []
        while len(row) < S:
            row += [rng.choice([-1, len(ids) + len(row), 3, 5])] * rng.randint(1, max(2, S // 4))
        row = row[:S]
        if shuffled:
            rng.shuffle(row)
        ids.append(row)
    return torch.tensor(ids, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(causal=True), dict(causal=True, prefix=True), dict(docs=True),
                                dict(docs=True, causal=True, prefix=True, bias=True, softcap=20.0), dict(bias=True),
                                dict(bias=True, causal=True), dict(softcap=8.0, causal=True)], ids=str)
def test_long(cuda_lib, D, kw):
    """More than 148 units and more than 32 KV tiles a walk; heads that are runs of their own and packed ones."""
    import torch
    for S, H, Hk in ((4700, 8, 2), (4429, 6, 6)):
        g, rng = torch.Generator(device="cuda").manual_seed(S), random.Random(S + D)
        q, k, v = _rand((2, H, S, D), g, 2.0), _rand((2, Hk, S, D), g), _rand((2, Hk, S, D), g)
        a = {n: x for n, x in kw.items() if n in ("causal", "softcap")}
        if kw.get("docs"):
            a["q_doc"] = a["kv_doc"] = _docs(rng, 2, S)
        if kw.get("prefix"):
            a["prefix"] = torch.tensor([600, 4200], dtype=torch.int32, device="cuda")
        if kw.get("bias"):
            a["slopes"] = torch.tensor([2.0 ** (-1.5 * (h + 1)) for h in range(H)], device="cuda")
        _check(cuda_lib, q, k, v, **a)


@pytest.mark.parametrize("seed", range(40))
def test_random_calls(cuda_lib, seed):
    import torch
    rng = random.Random(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    D, Hk = rng.choice([64, 128]), rng.choice([1, 2, 3])
    H, B = Hk * rng.choice([1, 2, 5]), rng.choice([1, 2, 3])
    S_kv = rng.choice([rng.randint(1, 300), rng.randint(300, 3000), rng.randint(3000, 9000)])
    S_q = rng.choice([1, rng.randint(1, 40), rng.randint(1, 700), min(S_kv, 1500)])
    q, k, v = _rand((B, H, S_q, D), g, rng.choice([0.5, 2.0])), _rand((B, Hk, S_kv, D), g), _rand((B, Hk, S_kv, D), g)
    a = dict(softcap=rng.choice([0.0, 0.0, 2.0, 30.0]), causal=rng.random() < 0.6)
    if a["causal"] and rng.random() < 0.5:
        a["prefix"] = torch.tensor([rng.randint(-5, S_kv + 200) for _ in range(B)], dtype=torch.int32, device="cuda")
    if rng.random() < 0.5:
        a["q_start"] = torch.tensor([rng.randint(-S_q, S_kv + 100) for _ in range(B)], dtype=torch.int32, device="cuda")
    if rng.random() < 0.4:
        a["slopes"] = torch.tensor([rng.choice([0.0, 0.01, 0.3, -0.002]) for _ in range(H)], device="cuda")
    if rng.random() < 0.5:
        a["q_doc"], a["kv_doc"] = _docs(rng, B, S_q, rng.random() < 0.3), _docs(rng, B, S_kv, rng.random() < 0.3)
    _check(cuda_lib, q, k, v, **a)


@pytest.mark.parametrize("D", [64, 128])
def test_what_earlier_calls_left_behind_does_not_matter(cuda_lib, D):
    """Shared and tensor memory full of NaN from the call before: the results are bit for bit those after a clean one."""
    import torch
    g, rng = torch.Generator(device="cuda").manual_seed(D), random.Random(D)
    S, H = 2200, 6
    q, k, v = (_rand((2, H, S, D), g) for _ in range(3))
    bad = torch.full_like(q, float("nan"))
    doc = _docs(rng, 2, S)
    calls = [dict(), dict(causal=True), dict(slopes=torch.full((H,), 0.1, device="cuda")),
             dict(slopes=torch.full((H,), 0.1, device="cuda"), causal=True), dict(q_doc=doc, kv_doc=doc),
             dict(q_doc=doc, kv_doc=doc, causal=True, softcap=5.0)]
    for kw in calls:
        for rows in (S, 40, 1):
            a = dict(kw, q_doc=doc[:, :rows].contiguous()) if "q_doc" in kw else kw
            qr, br = q[:, :, :rows].contiguous(), bad[:, :, :rows].contiguous()
            cuda_lib.masked_attention(qr, k, v)
            want = cuda_lib.masked_attention(qr, k, v, **a)
            for _ in range(3):
                cuda_lib.masked_attention(bad, bad, bad)
                cuda_lib.masked_attention(br, bad, bad)
                got = cuda_lib.masked_attention(qr, k, v, **a)
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (list(kw), rows)
