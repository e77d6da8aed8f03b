"""fp64 definitions of the operators around a block's attention: root-mean-square norm with the
residual's addition, rotary positions, and attention with capped scores, a distance bias and
causal, prefix and document masks.  Plain loops over rows and heads; no GPU, no torch."""

from __future__ import annotations

import numpy as np


def rms_norm(x, weight=None, residual=None, eps=1e-6):
    """(y, h): h = x + residual, y = h * weight / sqrt(mean(h^2) + eps) along the last axis."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    return y, h


def rope(x, pos, freqs, axis_pairs, interleaved, magnitude=1.0, weight=None, eps=1e-6):
    """x [B, S, H, D] -> [B, H, S, D]: norm over D (with a weight), then rotation of the first
    2 * len(freqs) elements; pos [B, S, axes] integers.  Whole turns are dropped in 128-bit integers."""
    x = np.asarray(x, np.float64)
    B, S, H, D = x.shape
    if weight is not None:
        x, _ = rms_norm(x, weight, eps=eps)
    y = np.moveaxis(x, 2, 1).copy()
    n = len(freqs)
    axis = np.repeat(np.arange(len(axis_pairs)), axis_pairs)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        # the angle as a fraction of a turn: position times the frequency's exact ratio, modulo one turn
        num, den = (float(freqs[i]) / (2 * np.pi)).as_integer_ratio()
        turn = np.array([[(int(p) * num % den) / den for p in row] for row in pos[..., axis[i]]])
        c, s = magnitude * np.cos(2 * np.pi * turn)[:, None], magnitude * np.sin(2 * np.pi * turn)[:, None]
        u, v = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    return y


def masked_attention(q, k, v, scale, softcap=0.0, slopes=None, causal=False, q_start=None, prefix=None, q_doc=None,
                     kv_doc=None):
    """(out, lse) row by row over the allowed keys only (the others are never touched)."""
    B, H, S_q, D = q.shape
    H_kv, S_kv = k.shape[1], k.shape[2]
    out = np.zeros((B, H, S_q, D))
    lse = np.full((B, H, S_q), -np.inf)
    j = np.arange(S_kv)
    for b in range(B):
        start = S_kv - S_q if q_start is None else int(q_start[b])
        for i in range(S_q):
            ok = np.ones(S_kv, bool)
            if causal:
                ok &= (j <= start + i) | (j < (0 if prefix is None else int(prefix[b])))
            if q_doc is not None:
                ok &= (kv_doc[b] == q_doc[b, i]) & (q_doc[b, i] >= 0)
            n = np.nonzero(ok)[0]
            if not n.size:
                continue
            for h in range(H):
                hk = h // (H // H_kv)
                s = (k[b, hk, n] @ q[b, h, i]) * scale
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s - float(slopes[h]) * np.abs(start + i - n)
                m = s.max()
                p = np.exp(s - m)
                out[b, h, i] = (p @ v[b, hk, n]) / p.sum()
                lse[b, h, i] = m + np.log(p.sum())
    return out, lse
