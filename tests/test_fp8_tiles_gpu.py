"""The 8-bit product where each CTA, or CTA pair, works through several tiles, in every kernel that
it chooses from, and reductions of tens of thousands, against 64 bits (needs a B200).

Tolerances: fp8_ref.product_error for the sums, GELU within 2^-18 of its value and 3e-8 below
z = -4.4 (tests/test_fp8_gelu_gpu.py) with |GELU'| <= 1.13, half a step of the output's type."""
import pytest
import torch

import fp8_ref as R
from test_fp8_gpu import mlp_expected, mlp_weights
from test_norm_gpu import draw, near_border, params

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")
BF, FP, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24


def _rs():
    import free_vit_token_b200 as rs
    return rs


def operands(M, N, K, seed):
    rs = _rs()
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(M, K, generator=g, device=dev).add_(0.1).to(BF)
    w = (torch.randn(N, K, generator=g, device=dev) * 0.05).to(BF)
    return rs.rs_fp8_quantize(x)[0], rs.rs_fp8_quantize(w)[0]


def products(a, b):
    """A B^T of the stored values and its error bound, rows in chunks."""
    bv = R.stored(b)
    z, d = [], []
    for r in range(0, a.rows, 8192):
        n = min(8192, a.rows - r)
        at = R.scale_index(a.rows, a.K)[r:r + n].to(dev)
        av = a.q[r:r + n, :a.K].double() * R.spread(a.scales[at].long() - 127, a.K)
        z.append(av @ bv.T)
        d.append(R.product_error(av, bv))
    return torch.cat(z), torch.cat(d)


def gelu(z, d):
    y = R.gelu(z)
    return y, R.GELU_SLOPE * d + 2.0 ** -18 * y.abs() + torch.where(z < -4.3, 3e-8, 0.0)


def held(got, y, d):
    """got is y within d and its own rounding."""
    return bool(((got.double() - y).abs() <= d + R.HALF_STEP[got.dtype] * (y.abs() + d) + R.tiny(got.dtype)).all())


# tiles per CTA or pair on 148 SMs: 256 columns single 4.2 (and 2.1), pair 4.3 (2.1), 128 columns
# single 3.2, pair 3.2; K past 1024 takes pairs with GELU too
@pytest.mark.parametrize("M,N,K", [(20000, 1000, 384), (20000, 500, 200), (20000, 1000, 1100),
                                   (20001, 330, 1031), (60000, 120, 384), (60000, 120, 640),
                                   (60000, 77, 1100)])
def test_several_tiles(M, N, K):
    rs = _rs()
    a, b = operands(M, N, K, M + N + K)
    z, d = products(a, b)
    bias = draw(1, N, BF, 3)[0]
    for dtype in (BF, FP):
        resid = draw(M, N, dtype, 4)
        assert held(rs.rs_fp8_gemm(a, b, out_dtype=dtype), z, d)
        zb = z + bias.double()
        db = d + U * zb.abs()
        y, e = gelu(zb, db)
        assert held(rs.rs_fp8_gemm(a, b, bias=bias, gelu=True, out_dtype=dtype), y, e)
        y = zb + resid.double()
        assert held(rs.rs_fp8_gemm(a, b, bias=bias, resid=resid, out_dtype=dtype), y, db + U * y.abs())
    q = R.stored(rs.rs_fp8_gemm(a, b, out_dtype=E4))
    assert ((q - R.quantized(z)).abs() <= near_border(z, d)).all()
    y, e = gelu(zb, db)
    q = R.stored(rs.rs_fp8_gemm(a, b, bias=bias, gelu=True, out_dtype=E4))
    diff = (q - R.quantized(y)).abs()
    assert (diff <= near_border(y, e)).all() and (diff == 0).double().mean() > 0.99
    assert rs.rs_get_last_device_error() == 0


@pytest.mark.parametrize("M,N,K", [(300, 200, 50000), (4000, 2000, 20000), (20000, 120, 9000)])
def test_long_reductions(M, N, K):
    rs = _rs()
    a, b = operands(M, N, K, 5)
    z, d = products(a, b)
    for dtype in (BF, FP):
        assert held(rs.rs_fp8_gemm(a, b, out_dtype=dtype), z, d)
    # not by the bound's width alone: the errors of the additions do not all point one way
    got = rs.rs_fp8_gemm(a, b, out_dtype=FP).double()
    assert (got - z).norm() <= 2.0 ** -17 * z.norm()
    assert rs.rs_get_last_device_error() == 0


@pytest.mark.parametrize("M,N,K", [(50432, 384, 192), (50433, 776, 200)])
def test_weight_gradient_of_a_large_batch(M, N, K):
    rs = _rs()
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn(M, K, generator=g, device=dev).add_(0.1).to(BF)
    w = (torch.randn(N, K, generator=g, device=dev) * 0.05).to(BF)
    dy = (torch.randn(M, N, generator=g, device=dev) * 1e-3).to(BF)
    xt, wt = rs.rs_fp8_quantize(x, False, True)[1], rs.rs_fp8_quantize(w, False, True)[1]
    dx, dw, db = rs.rs_fp8_linear_backward(dy, xt, wt, bias=True, dw_dtype=FP)
    q = R.quantized(dy.double().t().contiguous())
    xv = R.stored(xt)
    assert held(dw, q @ xv.T, R.product_error(q, xv))
    del q, xv
    q, wv = R.quantized(dy.double()), R.stored(wt)
    assert held(dx, q @ wv.T, R.product_error(q, wv))
    # sums over rows: a thread's chain of 8 rows a tile, then threads and blocks
    assert ((db.double() - dy.double().sum(0)).abs() <= (M / 64 + 40) * U * dy.double().abs().sum(0)).all()
    assert rs.rs_get_last_device_error() == 0


@pytest.mark.parametrize("M,C,H", [(8000, 512, 2048), (8000, 1152, 1024)])
def test_mlp_of_several_tiles(M, C, H):
    rs = _rs()
    x = draw(M, C, BF, M + C)
    w1, b1, w2, b2 = mlp_weights(C, H, 5)
    gamma, beta = params(C, BF, 6)
    got = rs.rs_mlp_forward_fp8(x, w1, b1, w2, b2, gamma, beta)
    want, tol = mlp_expected(x, w1, b1, w2, b2, gamma, beta)
    assert ((got.double() - want).abs() <= tol).all()
    assert (got.double() - want).norm() <= 3e-3 * want.norm()
    assert rs.rs_get_last_device_error() == 0


@pytest.mark.parametrize("M,N,K", [(130, 200, 200), (130, 8, 200), (20001, 330, 200), (20001, 1000, 1100)])
def test_8_bit_output_leaves_the_rest_alone(M, N, K):
    """Bytes past the row's last 16, rows past the last and scale bytes of neither row nor block."""
    rs = _rs()
    a, b = operands(M, N, K, 1)
    want = rs.rs_fp8_gemm(a, b, out_dtype=E4)
    ld = -(-N // 16) * 16
    buf = torch.full((M + 2, ld + 48), 0x55, dtype=torch.uint8, device=dev)
    sc = torch.full((rs.rs_fp8_scale_bytes(M, N),), 0x55, dtype=torch.uint8, device=dev)
    out = rs.Fp8(buf[1:M + 1, 16:16 + ld].view(E4), sc, M, N)
    rs.rs_fp8_gemm(a, b, out=out)
    assert torch.equal(R.stored(out), R.stored(want))
    assert (buf[0] == 0x55).all() and (buf[M + 1] == 0x55).all()
    assert (buf[:, :16] == 0x55).all() and (buf[:, 16 + ld:] == 0x55).all()
    live = torch.zeros_like(sc, dtype=torch.bool)
    live[R.scale_index(M, N).flatten().to(dev)] = True
    assert (sc[~live] == 0x55).all()


@pytest.mark.parametrize("M,C", [(130, 200), (3, 1160)])
def test_8_bit_norm_leaves_the_rest_alone(M, C):
    rs = _rs()
    x = draw(M, C, BF, 1)
    want = rs.rs_ln_quantize(x)
    buf = torch.full((M + 2, C + 56), 0x55, dtype=torch.uint8, device=dev)
    buf = buf[:, :(C + 56) // 16 * 16].contiguous()
    sc = torch.full((rs.rs_fp8_scale_bytes(M, C),), 0x55, dtype=torch.uint8, device=dev)
    out = rs.Fp8(buf[1:M + 1, 16:].view(E4), sc, M, C)
    rs.rs_ln_quantize(x, out=out)
    assert torch.equal(R.stored(out), R.stored(want))
    assert (buf[0] == 0x55).all() and (buf[M + 1] == 0x55).all()
    assert (buf[:, :16] == 0x55).all() and (buf[:, 16 + C:] == 0x55).all()
    live = torch.zeros_like(sc, dtype=torch.bool)
    live[R.scale_index(M, C).flatten().to(dev)] = True
    assert (sc[~live] == 0x55).all()
