"""Fit the polynomials that the rotary kernel evaluates cosines and sines with.

The kernel takes whole and quarter turns off in integers, so that the angle left is pi x with |x| <= 1/4.
sin(pi x) = x p(x^2) and cos(pi x) = q(x^2), p and q the polynomials of degree 4 closest in relative error on
[0, 1/16], found by iteratively reweighted least squares (Lawson's method), rounded to float32 (the constant of q
is exactly 1 then: cos(0) = 1).

Run:  python long_sequence_attention_b200/csrc/fit_rope_poly.py
"""

import numpy as np


def fit(f, degree: int, iters: int = 300):
    t = (1.0 - np.cos(np.linspace(0.0, np.pi, 4001))) / 32.0
    y = f(np.sqrt(np.maximum(t, 1e-14)))
    a = np.vander(t * 16.0, degree + 1, increasing=True) / y[:, None]
    w = np.ones_like(t)
    for _ in range(iters):
        sw = np.sqrt(w)
        c = np.linalg.lstsq(a * sw[:, None], sw, rcond=None)[0]
        e = np.abs(a @ c - 1.0)
        w = w * e / e.max() + 1e-12
        w /= w.mean()
    return c * 16.0 ** np.arange(degree + 1), e.max()


def check(ps, pc):
    """Largest absolute error of the float32 evaluation, in units of 2^-24."""
    f = np.float32
    x = np.linspace(-0.25, 0.25, 400001).astype(f)
    t = (x * x).astype(f)
    out = []
    for c, ref in ((ps, np.sin), (pc, np.cos)):
        r = np.full_like(x, c[-1])
        for k in c[-2::-1]:
            r = (r.astype(np.float64) * t + k).astype(f)           # one fma
        if ref is np.sin:
            r = (x * r).astype(f)
        out.append(np.abs(r.astype(np.float64) - ref(np.pi * x.astype(np.float64))).max() * 2.0 ** 24)
    return out


if __name__ == "__main__":
    s, es = fit(lambda x: np.sin(np.pi * x) / x, 4)
    c, ec = fit(lambda x: np.cos(np.pi * x), 4)
    s, c = s.astype(np.float32), c.astype(np.float32)
    print(f"relative error: sin {es:.2e}, cos {ec:.2e}; float32, in 2^-24: {check(s, c)}")
    print("sin", [float(v) for v in s])
    print("cos", [float(v) for v in c])
