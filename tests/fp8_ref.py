"""Layer norm and 8-bit blocks in 64 bits, from their definitions, for the tests: no code
shared with the library. Works on any device."""
import math

import torch

F64 = torch.float64
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24,
             torch.float8_e4m3fn: 2.0 ** -4}


def tiny(dtype):
    """Half the spacing of the type's subnormals."""
    return {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}[dtype]


def e4m3_step(v):
    """Spacing of e4m3 at |v|: 2^(floor(log2 |v|) - 3), from 2^-6 down 2^-9."""
    _, k = torch.frexp(v.abs().clamp(min=2.0 ** -6))
    return torch.ldexp(torch.ones_like(v), k - 4)


def e4m3(v):
    """Nearest e4m3 value, ties to even (|v| <= 448)."""
    s = e4m3_step(v)
    return torch.round(v / s) * s


def block_exponents(x):
    """[R, K] -> [R, ceil(K / 128)]: the least e >= -127 with max |x| <= 448 * 2^e over a
    block's finite values."""
    R, K = x.shape
    KB = -(-K // 128)
    p = torch.zeros(R, KB * 128, dtype=F64, device=x.device)
    p[:, :K] = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    a = p.view(R, KB, 128).abs().amax(-1)
    m, k = torch.frexp(a / 448.0)           # a / 448 = m 2^k, 1/2 <= m < 1
    e = torch.where(m == 0.5, k - 1, k).to(torch.int64)
    # a / 448 is rounded: settle the two neighbours exactly
    e = torch.where(448.0 * torch.exp2(e.double()) < a, e + 1, e)
    e = torch.where(448.0 * torch.exp2(e.double() - 1) >= a, e - 1, e)
    e = torch.where(a == 0, torch.full_like(e, -127), e)
    return e.clamp(min=-127)


def spread(e, K):
    """Block exponents to a factor 2^e per value."""
    return torch.exp2(e.double()).repeat_interleave(128, 1)[:, :K]


def quantized(x):
    """The values x [R, K] (64 bits) takes in 8-bit blocks; infinities and NaN become NaN."""
    f = spread(block_exponents(x), x.shape[1])
    fin = torch.isfinite(x)
    v = e4m3(torch.where(fin, x, torch.zeros_like(x)) / f) * f
    return torch.where(fin, v, torch.full_like(v, math.nan))


def scale_index(rows, K):
    """Place of every (row, block) scale byte."""
    r = torch.arange(rows)[:, None]
    j = torch.arange(-(-K // 128))[None, :]
    return (r // 128 * (-(-K // 512)) + j // 4) * 512 + 16 * (r % 32) + 4 * (r // 32 % 4) + j % 4


def stored(t):
    """The values an Fp8 stands for, in 64 bits."""
    at = scale_index(t.rows, t.K).to(t.scales.device)
    return t.q[:, :t.K].double() * spread(t.scales[at].long() - 127, t.K)


def layer_norm(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    var = (x - mean).square().mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt(var + eps)
    xh = (x - mean) * rstd
    y = xh
    if gamma is not None:
        y = y * gamma.double()
    if beta is not None:
        y = y + beta.double()
    return y, mean, rstd, xh


def layer_norm_grad(dy, x, gamma, eps, dres=None):
    _, _, rstd, xh = layer_norm(x, None, None, eps)
    dy = dy.double()
    w = dy if gamma is None else dy * gamma.double()
    dx = rstd * (w - w.mean(-1, keepdim=True) - xh * (w * xh).mean(-1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
    return dx, (dy * xh).sum(0), dy.sum(0)


def gelu(z):
    return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))


def product_error(aq, bq):
    """Bound of the fp32 accumulation's error of aq bq^T (stored values, which multiply exactly):
    an instruction adds 32 products to the accumulator and loses at most 2^-23 of the magnitudes
    it holds per addition, K / 32 instructions after one another, 5 levels within each."""
    K = aq.shape[1]
    return (-(-K // 32) + 5) * 2.0 ** -23 * (aq.abs() @ bq.abs().T)


GELU_ERR = 1.6e-5   # |GELU error| of the epilogue's polynomials (1.5e-5 near zero, 1.1e-6 beyond)
GELU_SLOPE = 1.13   # the largest |GELU'|
