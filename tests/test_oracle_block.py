"""CPU pins of oracle/block.py: closed forms, torch's fp64 operators and invariants."""

import numpy as np
import pytest
import torch

import oracle
from oracle import block


def test_norm_closed_forms():
    y, h = block.rms_norm([[3.0, 4.0]], eps=0.0)
    np.testing.assert_allclose(y, [[3 / np.sqrt(12.5), 4 / np.sqrt(12.5)]], rtol=1e-15)
    y, h = block.rms_norm([[1.0, -1.0]], weight=[2.0, 3.0], residual=[[1.0, -1.0]], eps=0.0)
    np.testing.assert_allclose(y, [[2.0, -3.0]], rtol=1e-15)
    np.testing.assert_array_equal(h, [[2.0, -2.0]])
    assert np.all(block.rms_norm(np.zeros((2, 5)))[0] == 0.0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_complex_turn(interleaved):
    r = np.random.default_rng(0)
    B, S, H, D, rot = 2, 5, 3, 16, 12
    x, pos = r.standard_normal((B, S, H, D)), r.integers(-50, 50, (B, S, 2))
    f = r.uniform(0.01, 3.0, rot // 2)
    y = block.rope(x, pos, f, [2, 4], interleaved)
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    ang = np.concatenate([pos[..., :1] * f[:2], pos[..., 1:] * f[2:]], -1)[:, :, None]
    z = (x[..., lo] + 1j * x[..., hi]) * np.exp(1j * ang)
    np.testing.assert_allclose(y[..., lo] + 1j * y[..., hi], np.moveaxis(z, 2, 1), atol=1e-12)
    np.testing.assert_array_equal(y[..., rot:], np.moveaxis(x, 2, 1)[..., rot:])


def test_rope_scores_depend_on_distance_only():
    r = np.random.default_rng(1)
    q, k = r.standard_normal((2, 1, 1, 1, 8))
    f = [1.0, 0.1, 0.01, 0.001]
    at = lambda x, p: block.rope(x, np.array([[[p]]]), f, [4], False)[0, 0, 0]
    np.testing.assert_allclose(at(q, 7) @ at(k, 3), at(q, 2000000007) @ at(k, 2000000003), atol=1e-9)


def test_masked_attention_against_the_plain_oracle_and_torch():
    r = np.random.default_rng(2)
    q, k, v = (r.standard_normal((1, 2, 9, 4)) for _ in range(3))
    o, l = block.masked_attention(q, k, v, 0.5)
    ro, rl = oracle.attention(q, k, v, 0.5)
    np.testing.assert_allclose(o, ro, atol=1e-13)
    np.testing.assert_allclose(l, rl, atol=1e-13)
    t = [torch.from_numpy(x) for x in (q, k, v)]
    ref = torch.nn.functional.scaled_dot_product_attention(*t, is_causal=True, scale=0.5).numpy()
    np.testing.assert_allclose(block.masked_attention(q, k, v, 0.5, causal=True)[0], ref, atol=1e-13)
    # documents cut the sequence into independent attentions; padding is empty
    doc = np.array([[0, 0, 0, 5, 5, 5, 5, -1, -1]])
    o, l = block.masked_attention(q, k, v, 0.5, q_doc=doc, kv_doc=doc)
    np.testing.assert_allclose(o[:, :, 3:7], oracle.attention(q[:, :, 3:7], k[:, :, 3:7], v[:, :, 3:7], 0.5)[0], atol=1e-13)
    assert np.all(o[:, :, 7:] == 0) and np.all(l[:, :, 7:] == -np.inf)


def test_masked_attention_cap_bias_prefix_closed_forms():
    q = np.array([[[[2.0], [2.0]]]])
    k = np.array([[[[1.0], [-1.0], [3.0]]]])
    v = np.array([[[[1.0], [10.0], [100.0]]]])
    # positions 1, 2 (of 3); capped at 1.5, slope 0.25
    s = 1.5 * np.tanh(np.array([2.0, -2.0, 6.0]) / 1.5)
    for i, pos in enumerate((1, 2)):
        e = np.exp(s - 0.25 * np.abs(pos - np.arange(3)))
        e[pos + 1:] = 0.0
        o, l = block.masked_attention(q, k, v, 1.0, softcap=1.5, slopes=[0.25], causal=True)
        np.testing.assert_allclose(o[0, 0, i, 0], (e @ v[0, 0, :, 0]) / e.sum(), rtol=1e-14)
        np.testing.assert_allclose(l[0, 0, i], np.log(e.sum()), rtol=1e-14)
    full = block.masked_attention(q, k, v, 1.0)
    seen = block.masked_attention(q, k, v, 1.0, causal=True, q_start=[-5], prefix=[3])
    np.testing.assert_allclose(seen[0], full[0], rtol=1e-14)
    assert np.all(block.masked_attention(q, k, v, 1.0, causal=True, q_start=[-5])[1] == -np.inf)
