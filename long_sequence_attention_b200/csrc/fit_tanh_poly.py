"""Fit the polynomials that the masked attention uses to cap scores by a tanh.

The kernel evaluates tanh(x) = x * p(x^2) on the FMA pipe (the special-function unit is busy with the softmax's
exponentials).  p is the polynomial closest to tanh(sqrt(t)) / sqrt(t) in relative error on [0, T], found by
iteratively reweighted least squares (Lawson's method) and rounded to float32: degree 3 for |x| <= 1/2 (T = 1/4),
the usual case, and degree 5 for |x| <= 1.  Scores beyond the cap take the exact formula.

Run:  python long_sequence_attention_b200/csrc/fit_tanh_poly.py
"""

import numpy as np


def fit(T: float, degree: int, iters: int = 400):
    t = (1.0 - np.cos(np.linspace(0.0, np.pi, 4001))) / 2.0 * T
    x = np.sqrt(np.maximum(t, 1e-12))
    y = np.tanh(x) / x
    a = np.vander(t / T, degree + 1, increasing=True) / y[:, None]
    w = np.ones_like(t)
    for _ in range(iters):
        sw = np.sqrt(w)
        c = np.linalg.lstsq(a * sw[:, None], sw, rcond=None)[0]
        e = np.abs(a @ c - 1.0)
        w = w * e / e.max() + 1e-12
        w /= w.mean()
    return c / T ** np.arange(degree + 1), e.max()


if __name__ == "__main__":
    for T, degree in ((0.25, 3), (1.0, 5)):
        c, err = fit(T, degree)
        print(f"|x| <= {T ** 0.5}: degree {degree}, max relative error {err:.2e}")
        print("  ", ", ".join(f"{float(v)!r}f" for v in c.astype(np.float32)))
