"""dit_rope_qk against the fp64 definition: layouts, partial heads, axes, far positions, packed
inputs, the norm, and the E4M3 blocks that the block-scaled attention reads."""

import numpy as np
import pytest

from oracle import block, fp8

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _bf16(shape, seed, scale=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _bound(x, pos, freqs, axis_pairs, interleaved, magnitude, w):
    """Error of one result in fp32, before its last rounding: the pair's length times the angle's and
    the arithmetic's errors.  Angle: the frequency in turns has two fp64 roundings here and two in the
    definition (2^-51 position * freq in all); the fraction is cut to 2^-32 turns and rounded to fp32 (pi U32);
    sincospi 2 ulps (4 U32), the magnitude and three products and sums (5 U32); the norm (D = 128: 4 in a
    lane, 5 steps, halved, plus rsqrt and two products: 12 U32)."""
    B, S, H, D = x.shape
    n = len(freqs)
    z = np.moveaxis(np.abs(block.rms_norm(x, w)[0] if w is not None else x), 2, 1).copy()
    p = np.abs(np.repeat(pos.astype(np.float64), axis_pairs, -1)) * np.abs(freqs)
    lo, hi = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    r = np.hypot(z[..., lo], z[..., hi]) * abs(magnitude) * (24 * U32 + p[:, None] * 2.0 ** -51)
    e = z * 12 * U32
    e[..., lo], e[..., hi] = r, r
    return e


def _run(lsa, q, k, pos, freqs, per, inter, mag, wq, wk, out):
    import torch
    q8 = lsa.rope_qk(q, k, torch.from_numpy(pos).cuda(), torch.from_numpy(freqs).cuda(), q_weight=wq, k_weight=wk,
                     axis_pairs=per, interleaved=inter, magnitude=mag, out_dtype=getattr(torch, out))
    pos = np.broadcast_to(pos if pos.ndim == 3 else pos[..., None], (q.shape[0], q.shape[1], len(per)))
    for x, w, y, d in ((q, wq, q8[0], q8[2]), (k, wk, q8[1], q8[3])):
        if x is None:
            assert y is None and d is None
            continue
        xn, wn = _np(x), None if w is None else _np(w)
        ref = block.rope(xn, pos, freqs, per, inter, mag, wn)
        e = _bound(xn, pos, freqs, per, inter, mag, wn)
        assert y.shape == ref.shape and y.is_contiguous()
        if d is None:
            assert np.all(np.abs(_np(y) - ref) <= np.abs(ref) * 2.0 ** -8 + e * (1 + 2.0 ** -8) + 1e-37)
            continue
        c, S = fp8.e4m3_decode(y.cpu().numpy()).astype(np.float64), ref.shape[2]
        for i in range(-(-S // 128)):
            sl = slice(128 * i, min(S, 128 * (i + 1)))
            amax = np.abs(ref[:, :, sl]).max((2, 3))
            dn = _np(d)[:, :, i]
            assert np.all(np.abs(dn - amax / 448.0) <= amax / 448.0 * 2.0 ** -19 + e[:, :, sl].max((2, 3)) / 448.0)
            back = c[:, :, sl] * dn[:, :, None, None]
            step = np.maximum(np.abs(ref[:, :, sl]) * 2.0 ** -4, dn[:, :, None, None] * 2.0 ** -10) * 1.001
            assert np.all(np.abs(back - ref[:, :, sl]) <= step + 2 * e[:, :, sl] + amax[:, :, None, None] * 2.0 ** -19)
    return q8


def _freqs(n, seed=0):
    return np.exp(np.random.default_rng(seed).uniform(np.log(1e-6), np.log(1.5), n))


SHAPES = [(1, 1, 1, 1, 64), (2, 3, 5, 2, 128), (3, 127, 2, 1, 64), (1, 129, 3, 3, 128), (2, 300, 6, 2, 64),
          (1, 513, 24, 4, 128), (8, 1, 24, 24, 128)]


@pytest.mark.parametrize("B,S,H,Hk,D", SHAPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("out", ["bfloat16", "uint8"])
def test_shapes_layouts_types(cuda_lib, B, S, H, Hk, D, inter, out):
    import torch
    r = np.random.default_rng(S * 7 + H)
    for rot, axes, norm, packed in ((D, 3, True, True), (D // 2, 1, False, False), (48, 2, True, False)):
        per = [rot // 2] if axes == 1 else ([rot // 4, rot // 2 - rot // 4] if axes == 2 else [2, 6, rot // 2 - 8])
        pos = r.integers(-5, 5000, (B, S, axes)).astype(np.int32)
        if packed:
            qkv = _bf16((B, S, H + 2 * Hk, D), S)
            q, k = qkv[:, :, :H], qkv[:, :, H:H + Hk]
        else:                                        # already head-major: a transposed view
            q, k = (_bf16((B, h, S, D), S + h, 3.0).transpose(1, 2) for h in (H, Hk))
        wq, wk = (_bf16((D,), 90), _bf16((D,), 91)) if norm else (None, _bf16((D,), 92))
        _run(cuda_lib, q, k, pos, _freqs(rot // 2), per, inter, 1.25 if norm else 1.0, wq, wk, out)


@pytest.mark.parametrize("rot", [2, 6, 50, 126])
def test_any_even_part_of_an_interleaved_head(cuda_lib, rot):
    q, k = _bf16((2, 9, 3, 128), 1), _bf16((2, 9, 2, 128), 2)
    pos = np.arange(9, dtype=np.int32)[None]
    for out in ("bfloat16", "uint8"):
        _run(cuda_lib, q, k, pos, _freqs(rot // 2), [rot // 2], True, 1.0, None, None, out)


def test_far_and_negative_positions(cuda_lib):
    pos = np.array([[[0], [1], [-1], [2 ** 24 + 1], [10 ** 9 + 7], [2 ** 31 - 1], [-2 ** 31], [-123456789]]], np.int32)
    q, k = _bf16((1, 8, 2, 64), 3), _bf16((1, 8, 1, 64), 4)
    f = np.concatenate([[1.0, 0.0, -0.7, 2 * np.pi, 100.0], _freqs(27, 1)])
    _run(cuda_lib, q, k, pos, f, [32], False, 1.0, None, None, "bfloat16")


def test_queries_alone_shared_positions_and_zero_rows(cuda_lib):
    import torch
    q = _bf16((2, 130, 3, 128), 5)
    pos = np.arange(130, dtype=np.int32)[None]
    _run(cuda_lib, q, None, pos, _freqs(64), [64], False, 1.0, None, None, "bfloat16")
    y, _, d, _ = _run(cuda_lib, q * 0, None, pos, _freqs(64), [64], True, 1.0, None, None, "uint8")
    assert torch.all(d == 0.0) and torch.all(y.view(torch.float8_e4m3fn).float() == 0)
    e = cuda_lib.rope_qk(q[:, :0], None, torch.zeros(1, 0, dtype=torch.int32, device="cuda"),
                         torch.ones(64, dtype=torch.float64, device="cuda"))
    assert e[0].shape == (2, 3, 0, 128)


def test_scaled_frequencies(cuda_lib):
    import torch
    f, m = cuda_lib.rope_frequencies(64, 10000.0, scaling="by_parts", factor=4.0, original_length=4096, device="cuda")
    base = 10000.0 ** (-np.arange(32) / 32)
    turns = 4096 * base / (2 * np.pi)
    got = f.cpu().numpy()
    assert np.allclose(got[turns > 32], base[turns > 32], rtol=1e-14)
    assert np.allclose(got[turns < 1], base[turns < 1] / 4, rtol=1e-14) and np.all((got <= base * (1 + 1e-14)) & (got >= base / 4.0001))
    assert abs(m - (0.1 * np.log(4.0) + 1)) < 1e-15
    f, m = cuda_lib.rope_frequencies(64, scaling="ntk", factor=8.0)
    assert f[0] == 1.0 and abs(f[-1].item() / (base[-1] / 8) - 1) < 1e-12 and m == 1.0
    f, _ = cuda_lib.rope_frequencies(64, scaling="linear", factor=8.0)
    assert np.allclose(f.numpy(), base / 8, rtol=1e-14)
    f, _ = cuda_lib.rope_frequencies(128, axis_pairs=[16, 24, 24])
    assert f.shape == (64,) and f[0] == f[16] == f[40] == 1.0


def test_stream_and_graph(cuda_lib):
    import torch
    q, k = _bf16((1, 300, 4, 128), 6), _bf16((1, 300, 2, 128), 7)
    pos = torch.arange(300, dtype=torch.int32, device="cuda")[None]
    f, _ = cuda_lib.rope_frequencies(128, device="cuda")
    call = lambda **kw: cuda_lib.rope_qk(q, k, pos, f, out_dtype=torch.uint8, **kw)
    want = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = call(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = call()
    q.neg_()
    pos.add_(1000)
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(call(), cap))
