"""Generates the constants of the 8-bit product's second GELU form (rs_gelu_logit.h).

GELU(z) = z Phi(z), with the normal CDF written as a logistic function: Phi(z) =
1 / (1 + 2^(-z Q(t))), t = min(z^2, T). z Q is odd like the logit of Phi, so Q is a polynomial in
z^2; it is fitted here to logit(Phi(z)) / (z ln 2) by Lawson's iteratively reweighted least
squares on Chebyshev nodes in t, weighted by the error it causes in GELU (z^2 Phi (1 - Phi)).
Past sqrt(T) Q keeps its last value, where 1 - Phi < 3e-7.

It costs half the FMAs of the polynomial form of rs_gelu_poly.h and three exponential-unit
instructions per two values instead, and needs no choice by range.

Run: python gen_gelu_logit.py > rs_gelu_logit.h
"""
import numpy as np
from scipy.special import log_ndtr, ndtr

T = 25.0
D = 3


def fit():
    n = 4000
    k = np.arange(n)
    t = (1.0 - np.cos(np.pi * (k + 0.5) / n)) / 2 * T
    z = np.sqrt(t)
    f = np.where(z > 1e-9, (log_ndtr(z) - log_ndtr(-z)) / np.maximum(z, 1e-12),
                 2 * np.sqrt(2 / np.pi)) / np.log(2.0)
    wt = z * z * ndtr(z) * ndtr(-z) + 1e-4
    V = np.vander(t, D + 1, increasing=True)
    w = np.ones(n)
    for _ in range(200):
        sw = np.sqrt(w) * wt
        c, *_ = np.linalg.lstsq(V * sw[:, None], f * sw, rcond=None)
        e = np.abs((V @ c - f) * wt)
        w = w * (e / e.max() + 1e-3)
        w /= w.sum()
    return c


def evaluate(c, z):
    """The kernel's form in float32 (exact 2^x and reciprocal)."""
    z = z.astype(np.float32)
    t = np.minimum(z * z, np.float32(T))
    p = np.full_like(z, np.float32(c[D]))
    for i in range(D - 1, -1, -1):
        p = p * t + np.float32(c[i])
    with np.errstate(over="ignore"):
        return z / (np.float32(1) + np.exp2((-z * p).astype(np.float32)))


if __name__ == "__main__":
    c = fit()
    z = np.linspace(-12, 12, 400001)
    err = np.abs(evaluate(c, z).astype(np.float64) - z * ndtr(z)).max()
    print("// Generated by gen_gelu_logit.py. GELU(z) = z / (1 + 2^(-z Q(min(z^2, T)))), Q of")
    print("// degree %d; max |error| %.2e in float32." % (D, err))
    print("#pragma once")
    print("#define RS_GELU_LOGIT_T %.1ff" % T)
    for i, v in enumerate(c):
        print("#define RS_GELU_LOGIT_Q%d %.9ef" % (i, v))
