"""GELU in the 8-bit products over every bf16 value: the lowest and largest ones, infinities and
NaN among them, beside one another in any order (needs a B200).

The operands are zero and the bias holds the values, so that the pre-activation is exact.
Tolerance: for |z| <= 4.4 the exponent z Q of the logistic form is fitted to 1e-6 and rounded a
few times at no more than 17.6: 1e-6 ln 2 + 3 * 2^-24 * 17.6 ln 2 = 2.9e-6 relative, 2^x and 1/x
add 2^-22 and 2^-23 of theirs, in all 3.3e-6 < 2^-18. Below z = -4.4 the form's own difference
from z Phi(z) is at most 1.8e-8 (z = -5.5), and GELU below 2.4e-5 times 1e-5 for the roundings of
an exponent of up to 25 there: 3e-8 covers both. Above 4.4 GELU is z (1 - 5e-6 ..): the error of
the second factor is at most that of Phi(-z), 1e-5 of 5.4e-6, and two roundings."""
import pytest
import torch

import fp8_ref as R
from test_norm_gpu import near_border

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")
BF, FP, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _rs():
    import free_vit_token_b200 as rs
    return rs


def every_bf16(shuffled):
    v = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    if shuffled:
        v = v[torch.randperm(1 << 16, generator=torch.Generator().manual_seed(7))]
    return v.view(BF).to(dev)


def bound(y, z):
    return 2.0 ** -18 * y.abs() + torch.where(z < -4.4, 3e-8, 0.0)


def check(got, z):
    """got [M, N] bf16 or fp32, every row GELU(z)."""
    want = R.gelu(z.double())
    one = got[0].double()
    bits = got.view(torch.int16 if got.dtype == BF else torch.int32)
    assert (bits == bits[:1]).all()
    fin = want.isfinite()
    assert torch.equal(one.isnan(), want.isnan())
    assert torch.equal(one[~fin & ~want.isnan()], want[~fin & ~want.isnan()])
    d = bound(want[fin], z[fin].double())
    tol = d + R.HALF_STEP[got.dtype] * (want[fin].abs() + d) + R.tiny(got.dtype)
    bad = (one[fin] - want[fin]).abs() > tol
    assert not bad.any(), (z[fin][bad][:4], one[fin][bad][:4], want[fin][bad][:4])


def zeros(rows, K):
    return _rs().rs_fp8_quantize(torch.zeros(rows, K, dtype=BF, device=dev))[0]


# one 128-column tile a CTA, 256 columns, a CTA pair
@pytest.mark.parametrize("M,K", [(5, 16), (300, 200), (300, 1040)])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shuffled", [False, True])
def test_gemm(M, K, dtype, shuffled):
    rs = _rs()
    z = every_bf16(shuffled)
    check(rs.rs_fp8_gemm(zeros(M, K), zeros(1 << 16, K), bias=z, gelu=True, out_dtype=dtype), z)
    assert rs.rs_get_last_device_error() == 0


@pytest.mark.parametrize("M,K", [(5, 16), (300, 200), (300, 1040)])
@pytest.mark.parametrize("shuffled", [False, True])
def test_gemm_to_blocks(M, K, shuffled):
    """One far negative value may not become its block's maximum."""
    rs = _rs()
    z = every_bf16(shuffled)
    q = rs.rs_fp8_gemm(zeros(M, K), zeros(1 << 16, K), bias=z, gelu=True, out_dtype=E4)
    got = R.stored(q)
    y = R.gelu(z.double())[None]
    want = R.quantized(y)
    fin = y.isfinite()
    y0 = torch.where(fin, y, torch.zeros_like(y))
    tol = near_border(y0, torch.where(fin, bound(y0, z.double()[None]), torch.zeros_like(y0)))
    for row in (got[:1], got[-1:]):
        assert torch.equal(row.isnan(), want.isnan())
        assert ((row - want)[fin].abs() <= tol[fin]).all()
    assert rs.rs_get_last_device_error() == 0


# a few rows in one launch, one and several CTAs to a reduction; and past them
@pytest.mark.parametrize("M,K", [(1, 16), (16, 300), (16, 2048), (40, 16)])
@pytest.mark.parametrize("shuffled", [False, True])
def test_linear(M, K, shuffled):
    rs = _rs()
    z = every_bf16(shuffled)
    x = torch.zeros(M, K, dtype=BF, device=dev)
    check(rs.rs_fp8_linear(x, zeros(1 << 16, K), bias=z, gelu=True), z)
    n = 8000                                     # up to 32 rows
    x = torch.zeros(32, K, dtype=BF, device=dev)
    check(rs.rs_fp8_linear(x, zeros(n, K), bias=z[-n:].contiguous(), gelu=True), z[-n:])
    assert rs.rs_get_last_device_error() == 0


def test_far_pre_activations_from_the_product():
    """The same values as sums of the product: 2^66, 2^100 and their negatives beside small ones."""
    rs = _rs()
    K, N = 128, 512
    x = torch.zeros(200, K, dtype=FP, device=dev)
    x[:, 0] = 1.0
    w = torch.zeros(N, K, dtype=FP, device=dev)
    e = torch.linspace(-3, 100, N, device=dev).round()
    w[:, 0] = torch.where(torch.arange(N, device=dev) % 3 == 0, torch.exp2(e), -torch.exp2(e))
    w[1::2, 0] = torch.linspace(-6, 6, N // 2, device=dev)
    a, b = rs.rs_fp8_quantize(x)[0], rs.rs_fp8_quantize(w)[0]
    z = R.stored(b)[:, 0]
    check(rs.rs_fp8_gemm(a, b, gelu=True, out_dtype=FP), z)
    check(rs.rs_fp8_gemm(a, b, gelu=True), z)
    check(rs.rs_fp8_linear(x[:7].to(BF), b, gelu=True), z)
