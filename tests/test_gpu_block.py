"""The norm, the rotary step and the attention as a block uses them one after another, captured as one graph too, and
what the Python helpers refuse."""

import numpy as np
import pytest

import oracle
from gpu_util import assert_bf16_parity, assert_fp8_parity, metrics
from oracle import block, fp8

pytestmark = pytest.mark.gpu


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _bf16(shape, seed, scale=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _block(lsa, st, fp8_attention):
    """stream + update -> norm -> projection -> norm and rotation of q and k -> attention; every stage's results."""
    import torch
    B, S, H, Hk, D = st["dims"]
    y, stream, _ = lsa.rms_norm(st["x"], st["w"], residual=st["r"])
    qkv = (y.view(B * S, -1) @ st["proj"]).view(B, S, H + 2 * Hk, D)
    v = qkv[:, :, H + Hk:].transpose(1, 2).contiguous()
    q, k, dq, dk = lsa.rope_qk(qkv[:, :, :H], qkv[:, :, H:H + Hk], st["pos"], st["freqs"], q_weight=st["wq"],
                               k_weight=st["wk"], interleaved=True, out_dtype=torch.uint8 if fp8_attention else None)
    if fp8_attention:
        v8, dv = lsa.quantize_fp8_blocks(v)
        return (y, stream, q, k, dq, dk, v8, dv) + lsa.attention_fp8_blocks(q, k, v8, dq, dk, dv)
    return (y, stream, q, k, v) + lsa.masked_attention(q, k, v, q_doc=st["doc"], kv_doc=st["doc"], softcap=20.0)


def _state(lsa, H, Hk, D, seed=0):
    import torch
    B, S, C = 2, 270, 320
    doc = torch.zeros(B, S, dtype=torch.int32, device="cuda")
    doc[0, 100:], doc[1, 250:] = 4, -1
    freqs, _ = lsa.rope_frequencies(D, device="cuda")
    return dict(dims=(B, S, H, Hk, D), x=_bf16((B, S, C), seed), r=_bf16((B, S, C), seed + 1, 2.0), w=_bf16((C,), seed + 2),
                proj=_bf16((C, (H + 2 * Hk) * D), seed + 3, C ** -0.5), wq=_bf16((D,), seed + 4), wk=_bf16((D,), seed + 5),
                pos=torch.arange(S, dtype=torch.int32, device="cuda")[None], freqs=freqs, doc=doc)


def test_bf16_block(cuda_lib):
    st = _state(cuda_lib, 6, 2, 64)
    y, stream, q, k, v, o, l = _block(cuda_lib, st, False)
    ref, h = block.rms_norm(_np(st["x"]), _np(st["w"]), _np(st["r"]))
    assert np.all(np.abs(_np(y) - ref) <= np.abs(ref) * 2.0 ** -7.9) and np.all(np.abs(_np(stream) - h) <= np.abs(h) * 2.0 ** -8)
    # head scores of a normed, rotated pair depend on the distance only through the rotation: row lengths are the norm's
    ro, rl = block.masked_attention(_np(q), _np(k), _np(v), 64 ** -0.5, softcap=20.0, q_doc=st["doc"].cpu().numpy(),
                                    kv_doc=st["doc"].cpu().numpy())
    assert_bf16_parity(metrics(_np(o), ro, _np(l), rl))
    assert np.all(_np(o)[1, :, 250:] == 0)


def test_e4m3_block(cuda_lib):
    st = _state(cuda_lib, 4, 4, 128, 20)
    y, stream, q, k, dq, dk, v8, dv, o, l = _block(cuda_lib, st, True)
    deq = [fp8.dequantize_per_block(c.cpu().numpy(), d.cpu().numpy()) for c, d in ((q, dq), (k, dk), (v8, dv))]
    ro, rl = oracle.attention(*deq, 128 ** -0.5)
    assert_fp8_parity(metrics(_np(o), ro, _np(l), rl))


@pytest.mark.parametrize("fp8_attention", [False, True])
def test_block_in_a_graph(cuda_lib, fp8_attention):
    import torch
    st = _state(cuda_lib, 4, 4, 128, 40)
    _block(cuda_lib, st, fp8_attention)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _block(cuda_lib, st, fp8_attention)
    for step in range(3):
        st["x"].copy_(_bf16(st["x"].shape, 60 + step))
        g.replay()
        want = _block(cuda_lib, st, fp8_attention)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert cuda_lib.dit_device_status() == 0


def test_refusals_on_gpu_tensors(cuda_lib):
    import torch
    lsa, z = cuda_lib, lambda *s, **k: torch.zeros(*s, device="cuda", **k)
    b16, i32 = torch.bfloat16, torch.int32
    x = z(4, 64, dtype=b16)
    bad = [lambda: lsa.rms_norm(x.half()), lambda: lsa.rms_norm(x.t()), lambda: lsa.rms_norm(x, z(64)),
           lambda: lsa.rms_norm(x, residual=z(4, 63, dtype=b16)), lambda: lsa.rms_norm(x, inplace=True),
           lambda: lsa.rms_norm(x, out_dtype=torch.float16), lambda: lsa.rms_norm(z(4, 0, dtype=b16))]
    q, pos, f = z(2, 5, 3, 64, dtype=b16), z(2, 5, dtype=i32), torch.ones(32, dtype=torch.float64, device="cuda")
    bad += [lambda: lsa.rope_qk(q.float(), None, pos, f), lambda: lsa.rope_qk(q, q[:1], pos, f),
            lambda: lsa.rope_qk(q, None, pos.long(), f), lambda: lsa.rope_qk(q, None, pos[:, :4].contiguous(), f),
            lambda: lsa.rope_qk(q, None, pos, f.float()), lambda: lsa.rope_qk(q, None, pos, f, axis_pairs=[16, 16]),
            lambda: lsa.rope_qk(q, None, pos, f, q_weight=z(32, dtype=b16)),
            lambda: lsa.rope_qk(q.transpose(2, 3), None, pos, f), lambda: lsa.rope_qk(q, None, pos.cpu(), f)]
    a = z(2, 4, 5, 64, dtype=b16)
    bad += [lambda: lsa.masked_attention(a, a, a[:, :2]), lambda: lsa.masked_attention(a, a.transpose(2, 3), a),
            lambda: lsa.masked_attention(a.half(), a, a), lambda: lsa.masked_attention(a, a, a, slopes=z(3)),
            lambda: lsa.masked_attention(a, a, a, causal=True, q_start=z(2)),
            lambda: lsa.masked_attention(a, a, a, q_doc=z(2, 5, dtype=i32)), lambda: lsa.masked_attention(a, a.cpu(), a)]
    for f_ in bad:
        with pytest.raises(ValueError):
            f_()
    refused = [lambda: lsa.masked_attention(a, a[:, :3].contiguous(), a[:, :3].contiguous()),
               lambda: lsa.masked_attention(a, a, a, prefix=z(2, dtype=i32)), lambda: lsa.masked_attention(a, a, a, softcap=-1.0),
               lambda: lsa.rms_norm(x, eps=-1.0), lambda: lsa.rms_norm(x, out_dtype=torch.uint8, group=64),
               lambda: lsa.rope_qk(q, None, pos, f[:12])]
    for f_ in refused:
        with pytest.raises(lsa.DitError):
            f_()
