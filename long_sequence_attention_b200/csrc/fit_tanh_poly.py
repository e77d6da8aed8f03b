"""Fit the polynomial that the masked attention uses to cap scores by a tanh.

For |x| <= 1 the kernel evaluates tanh(x) = x * p(x^2) on the FMA pipe (the special-function
unit is busy with the softmax's exponentials); p is the degree-5 polynomial closest to
tanh(sqrt(t)) / sqrt(t) in relative error on [0, 1], found by iteratively reweighted least
squares (Lawson's method), rounded to float32.  Scores beyond the cap take the exact formula.

Run:  python long_sequence_attention_b200/csrc/fit_tanh_poly.py [degree]
"""

import sys

import numpy as np


def fit(degree: int, iters: int = 400):
    t = (1.0 - np.cos(np.linspace(0.0, np.pi, 4001))) / 2.0
    x = np.sqrt(np.maximum(t, 1e-12))
    y = np.tanh(x) / x
    a = np.vander(t, degree + 1, increasing=True) / y[:, None]
    w = np.ones_like(t)
    for _ in range(iters):
        sw = np.sqrt(w)
        c = np.linalg.lstsq(a * sw[:, None], sw, rcond=None)[0]
        e = np.abs(a @ c - 1.0)
        w = w * e / e.max() + 1e-12
        w /= w.mean()
    return c, e.max()


if __name__ == "__main__":
    c, err = fit(int(sys.argv[1]) if len(sys.argv) > 1 else 5)
    print(f"max relative error {err:.3e}")
    for i, v in enumerate(c.astype(np.float32)):
        print(f"  c{i} = {float(v)!r}f")
