"""Generates the constants of the 8-bit products' GELU (rs_gelu_logit.h).

GELU(z) = z Phi(z), with the normal CDF written as a logistic function: Phi(z) =
1 / (1 + 2^(-z Q(z^2))). z Q is odd like the logit of Phi, so Q is a polynomial in t = z^2; it is
fitted here to logit(Phi(z)) / (z ln 2) on t < T by Lawson's iteratively reweighted least squares
on Chebyshev nodes in t, weighted by the relative error that it causes in GELU(-z),
z Phi(z) ln 2 per unit of Q. The degree is one whose leading coefficient is positive and whose Q
grows past T: then the exponent needs no bound and no choice by range. For z -> -inf, 2^(-z Q)
overflows and GELU vanishes (z = -inf itself gives -inf * 0, NaN, as z Phi(z) does); for z -> inf
it is z.

Run: python gen_gelu_logit.py > rs_gelu_logit.h
"""
import numpy as np
from scipy.special import log_ndtr, ndtr

T = 20.0
D = 9


def fit():
    n = 6000
    k = np.arange(n)
    t = (1.0 - np.cos(np.pi * (k + 0.5) / n)) / 2 * T
    z = np.sqrt(t)
    f = np.where(z > 1e-6, (log_ndtr(z) - log_ndtr(-z)) / np.maximum(z, 1e-12),
                 2 * np.sqrt(2 / np.pi)) / np.log(2.0)
    wt = z * ndtr(z)
    V = np.polynomial.chebyshev.chebvander(2 * t / T - 1, D)
    w = np.ones(n)
    for _ in range(400):
        sw = np.sqrt(w) * wt
        c, *_ = np.linalg.lstsq(V * sw[:, None], f * sw, rcond=None)
        e = np.abs((V @ c - f) * wt)
        w = w * (e / e.max() + 1e-4)
        w /= w.sum()
    c = np.polynomial.Chebyshev(c, domain=[0, T]).convert(kind=np.polynomial.Polynomial).coef
    far = np.polyval(c[::-1], np.linspace(T, 100 * T, 100000))
    assert c[D] > 0 and (np.diff(far) > 0).all()
    return c


def evaluate(c, z):
    """The kernel's form in float32 (exact 2^x and reciprocal)."""
    f = np.float32
    z = z.astype(f)
    with np.errstate(over="ignore", invalid="ignore"):
        t = z * z
        p = np.full_like(z, f(c[D]))
        for i in range(D - 1, -1, -1):  # the sum in float64 rounds once, as an FMA does
            p = (p.astype(np.float64) * t.astype(np.float64) + float(f(c[i]))).astype(f)
        x = -z * p
        return z * (f(1) / (f(1) + np.exp2(x.astype(np.float64)).astype(f)))


if __name__ == "__main__":
    c = fit()
    z = np.linspace(-12, 12, 960001).astype(np.float32)
    z = z[z != 0]
    want = z.astype(np.float64) * ndtr(z.astype(np.float64))
    err = np.abs(evaluate(c, z).astype(np.float64) - want)
    near = z >= -4.4
    print("// Generated by gen_gelu_logit.py. GELU(z) = z / (1 + 2^(-z Q(z^2))), Q of degree %d. In" % D)
    print("// float32 max |error| / |GELU| %.1e for z >= -4.4, max |error| %.1e below." %
          ((err[near] / np.abs(want[near])).max(), err[~near].max()))
    print("#pragma once")
    for i, v in enumerate(c):
        print("#define RS_GELU_LOGIT_Q%d %.9ef" % (i, v))
