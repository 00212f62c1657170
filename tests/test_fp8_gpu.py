"""Quantisation, the 8-bit product, the linear layer forward and backward and the MLP in 8 bits
against 64 bits (needs a B200). Quantisation is exact by definition (one rounding of an exact
value), so it is compared bit for bit; products carry fp8_ref.product_error and half a step of
the output's type."""
import ctypes

import pytest
import torch

import fp8_ref as R
from test_norm_gpu import draw, near_border, params, xh_error

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")
BF, HF, FP, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24


def _rs():
    import free_vit_token_b200 as rs
    return rs


def same(got, want):
    """Equal values, NaN where NaN."""
    return bool(((got == want) | (got.isnan() & want.isnan())).all())


# ------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("dtype", [BF, HF, FP], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 64), (2, 129), (7, 200), (128, 128), (129, 512),
                                 (395, 776), (513, 77), (1000, 1024), (9000, 40), (130, 2049)])
def test_quantize(M, K, dtype):
    rs = _rs()
    x = draw(M, K, dtype, M + K) * torch.logspace(-3, 3, M, device=dev)[:, None].to(dtype)
    want, want_t = R.quantized(x.double()), R.quantized(x.double().t().contiguous())
    q, qt, cs = rs.rs_fp8_quantize(x, True, True, True)
    assert same(R.stored(q), want) and same(R.stored(qt), want_t)
    tol = (M / 64 + 40) * U * x.double().abs().sum(0)
    assert ((cs.double() - x.double().sum(0)).abs() <= tol).all()
    assert same(R.stored(rs.rs_fp8_quantize(x)[0]), want)
    assert same(R.stored(rs.rs_fp8_quantize(x, False, True)[1]), want_t)


def test_quantize_borders_extremes_and_nonfinite():
    rs = _rs()
    x = torch.zeros(16, 384, device=dev)
    x[0, :128] = torch.linspace(-448, 448, 128)
    x[1, 5], x[1, 130], x[1, 260] = 448.0, 448.0001, 1.75 * 2.0 ** -60
    x[2, 0], x[2, 200] = 3.4028234e38, -3.4028234e38
    x[2, 1] = 1.0
    x[3, 0], x[3, 1] = 1e-40, -3e-42                     # subnormal
    x[4, :128] = torch.arange(128) * (2.0 ** -9 / 2) + 2.0 ** -9 / 4   # ties of the least values
    x[4, 0] = 448.0
    x[5, 3], x[5, 4] = float("inf"), 5.0
    x[6, 300], x[6, 301] = float("nan"), -7.0
    x[7, :] = float("-inf")
    x[8, 0] = -0.0
    v = torch.arange(256, dtype=torch.uint8, device=dev).view(E4).float()
    v = v[torch.isfinite(v)].sort().values
    x[9, :252] = torch.where(torch.arange(252, device=dev) % 126 == 0, 448.0, (v[1:253] + v[:252]) / 2)
    for dtype in (FP, BF):
        y = x.to(dtype)
        q, qt, _ = rs.rs_fp8_quantize(y, True, True)
        assert same(R.stored(q), R.quantized(y.double()))
        assert same(R.stored(qt), R.quantized(y.double().t().contiguous()))


def test_quantize_strided_unaligned_and_left_alone():
    rs = _rs()
    M, K = 150, 136
    for off, ld in ((0, 144), (1, 144), (3, 141), (8, 152)):
        buf = draw(M, ld, BF, off)
        x = buf.flatten()[off:off + (M - 1) * ld + K].as_strided((M, K), (ld, 1)) if off + K <= ld \
            else buf[:, :K]
        out, out_t = rs.rs._fp8_empty(M + 1, K + 40, dev), rs.rs._fp8_empty(K + 1, M + 40, dev)
        for o in (out, out_t):
            o.q.view(torch.uint8).fill_(0x55)
            o.scales.fill_(0x55)
        L, p = rs.lib(), lambda t: t.data_ptr()  # noqa: E731
        assert L.rs_fp8_quantize(p(x), x.stride(0), M, K, rs.RS_BF16, p(out.q), out.q.stride(0),
                                 p(out.scales), p(out_t.q), out_t.q.stride(0), p(out_t.scales), None,
                                 None, 0, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
        a = rs.Fp8(out.q[:M], out.scales, M, K)
        b = rs.Fp8(out_t.q[:K], out_t.scales, K, M)
        assert same(R.stored(a), R.quantized(x.double()))
        assert same(R.stored(b), R.quantized(x.double().t().contiguous()))
        qa, qb = out.q.view(torch.uint8), out_t.q.view(torch.uint8)
        assert (qa[M:] == 0x55).all() and (qa[:, -(-K // 16) * 16:] == 0x55).all()
        assert (qb[K:] == 0x55).all() and (qb[:, -(-M // 16) * 16:] == 0x55).all()


# ------------------------------------------------------------------ the product
def operands(M, N, K, seed, scale=1.0):
    rs = _rs()
    a = rs.rs_fp8_quantize(draw(M, K, BF, seed, 0.1, scale))[0]
    b = rs.rs_fp8_quantize(draw(N, K, BF, seed + 1, 0.0, 0.05))[0]
    return a, b


def epilogue_tol(a, b, bias, gelu, resid, dtype, R_=R):
    """(expected, tolerance) of rs_fp8_gemm's bf16 or fp32 output."""
    av, bv = R.stored(a), R.stored(b)
    z, d = av @ bv.T, R.product_error(av, bv)
    if bias is not None:
        z = z + bias.double()
        d = d + U * z.abs()
    if gelu:
        z, d = R.gelu(z), R.GELU_SLOPE * d + R.GELU_ERR + U * z.abs()
    if resid is not None:
        z = z + resid.double()
        d = d + U * z.abs()
    return z, d + R.HALF_STEP[dtype] * (z.abs() + d) + R.tiny(dtype)


SHAPES = [(1, 8, 1), (1, 256, 128), (3, 72, 200), (16, 2048, 2048), (64, 264, 96), (128, 64, 64),
          (129, 128, 384), (200, 192, 1000), (256, 512, 512), (300, 1000, 1032), (394, 768, 192),
          (1000, 320, 4096), (2500, 1024, 640), (5, 1000, 8192), (130, 130, 130)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(M, N, K):
    rs = _rs()
    a, b = operands(M, N, K, M + N + K)
    bias = draw(1, N, BF, 3)[0]
    resid = draw(M, N, BF, 4)
    for kw in (dict(), dict(bias=bias, gelu=True), dict(bias=bias, resid=resid)):
        got = rs.rs_fp8_gemm(a, b, **kw)
        want, tol = epilogue_tol(a, b, kw.get("bias"), kw.get("gelu", False), kw.get("resid"), BF)
        assert ((got.double() - want).abs() <= tol).all()
    got = rs.rs_fp8_gemm(a, b, out_dtype=FP)
    want, tol = epilogue_tol(a, b, None, False, None, FP)
    assert ((got.double() - want).abs() <= tol).all()
    acc = got.clone()
    rs.rs_fp8_gemm(a, b, resid=acc, out=acc)                 # accumulate in place
    assert ((acc.double() - 2 * want).abs() <= 2 * tol + 2 * U * want.abs()).all()
    assert torch.equal(rs.rs_fp8_gemm(a, b, out_dtype=FP), got)
    # 8-bit output: quantised from the fp32 result
    q = rs.rs_fp8_gemm(a, b, bias=bias, gelu=True, out_dtype=E4)
    av, bv = R.stored(a), R.stored(b)
    z = av @ bv.T + bias.double()
    d = R.GELU_SLOPE * (R.product_error(av, bv) + U * z.abs()) + R.GELU_ERR
    y = R.gelu(z)
    assert ((R.stored(q) - R.quantized(y)).abs() <= near_border(y, d)).all()
    assert rs.rs_get_last_device_error() == 0


@pytest.mark.parametrize("N,ld,off", [(77, 77, 0), (80, 83, 0), (80, 88, 1), (256, 256, 3), (1, 1, 0),
                                      (333, 336, 0)])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_gemm_output_rows_of_any_pitch(N, ld, off, dtype):
    rs = _rs()
    M, K = 140, 200
    a, b = operands(M, N, K, 5)
    flat = torch.full((off + (M + 1) * ld + 8,), 9.0, dtype=dtype, device=dev)
    out = flat[off:off + M * ld].view(M, ld)[:, :N]
    resid = draw(M, ld + 1, dtype, 6)[:, 1:1 + N]
    got = rs.rs_fp8_gemm(a, b, resid=resid, out=out)
    want, tol = epilogue_tol(a, b, None, False, resid, dtype)
    assert ((got.double() - want).abs() <= tol).all()
    assert (flat[:off] == 9).all() and (flat[off + M * ld:] == 9).all()
    assert (flat[off:off + M * ld].view(M, ld)[:, N:] == 9).all()


def test_gemm_scales_reach_their_rows_and_blocks():
    """Powers of two far apart, one per block: each must meet its own row, block and operand."""
    rs = _rs()
    M, N, K = 300, 520, 1100
    g = torch.Generator().manual_seed(1)
    ea = torch.randint(-20, 20, (M, 9), generator=g).to(dev)
    eb = torch.randint(-20, 20, (N, 9), generator=g).to(dev)
    x = draw(M, K, FP, 2) * R.spread(ea, K).float()
    w = draw(N, K, FP, 3) * R.spread(eb, K).float()
    a, b = rs.rs_fp8_quantize(x)[0], rs.rs_fp8_quantize(w)[0]
    got = rs.rs_fp8_gemm(a, b, out_dtype=FP)
    want, tol = epilogue_tol(a, b, None, False, None, FP)
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("ea,eb", [(-126, 100), (-122, 118), (118, -120), (0, -126)])
def test_gemm_scales_at_the_ends_of_their_range(ea, eb):
    """Scale bytes down to 0 (2^-127) and up to 2^112 in one operand."""
    rs = _rs()
    for M in (5, 300):
        x = draw(M, 300, FP, 2) * 2.0 ** ea
        w = draw(200, 300, FP, 3) * 2.0 ** eb
        a, b = rs.rs_fp8_quantize(x)[0], rs.rs_fp8_quantize(w)[0]
        assert same(R.stored(a), R.quantized(x.double()))
        got = rs.rs_fp8_gemm(a, b, out_dtype=FP)
        want, tol = epilogue_tol(a, b, None, False, None, FP)
        # results below fp32's normal range may be flushed to zero
        assert ((got.double() - want).abs() <= tol + 2.0 ** -126).all()


def test_norm_with_infinite_gamma():
    rs = _rs()
    x = draw(9, 256, BF, 1)
    gamma, beta = params(256, BF, 2)
    gamma[7] = float("inf")
    v = R.stored(rs.rs_ln_quantize(x, gamma, beta))
    assert v[:, 7].isnan().all() and not v[:, :7].isnan().any() and not v[:, 8:].isnan().any()
    g2 = gamma.clone()
    g2[7] = 0
    b2 = beta.clone()
    b2[7] = 0
    w = R.stored(rs.rs_ln_quantize(x, g2, b2))
    keep = [c for c in range(256) if c != 7]
    assert torch.equal(v[:, keep], w[:, keep])        # the block's scale is its finite values'


def test_gemm_nan_and_infinity_stay_in_their_row():
    rs = _rs()
    x, w = draw(200, 300, BF, 1), draw(150, 300, BF, 2)
    clean = rs.rs_fp8_gemm(rs.rs_fp8_quantize(x)[0], rs.rs_fp8_quantize(w)[0])
    x[5, 17], x[150, 299], w[70, 3] = float("nan"), float("inf"), float("-inf")
    a, b = rs.rs_fp8_quantize(x)[0], rs.rs_fp8_quantize(w)[0]
    got = rs.rs_fp8_gemm(a, b)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[5], bad[150], bad[:, 70] = True, True, True
    assert got[bad].isnan().all() and torch.equal(got[~bad], clean[~bad])
    q = R.stored(rs.rs_fp8_gemm(a, b, out_dtype=E4))
    assert q[bad].isnan().all() and not q[~bad].isnan().any()


def test_gemm_unwritten_scale_bytes_do_not_matter():
    """Scale bytes of rows and blocks that do not exist may hold anything, 0xFF (NaN) too."""
    rs = _rs()
    M, N, K = 130, 200, 200
    a, b = operands(M, N, K, 9)
    want = rs.rs_fp8_gemm(a, b)
    wq = R.stored(rs.rs_fp8_gemm(a, b, out_dtype=E4))
    for t in (a, b):
        live = torch.zeros_like(t.scales, dtype=torch.bool)
        live[R.scale_index(t.rows, t.K).flatten().to(dev)] = True
        t.scales[~live] = 0xFF
    assert torch.equal(rs.rs_fp8_gemm(a, b), want)
    assert torch.equal(R.stored(rs.rs_fp8_gemm(a, b, out_dtype=E4)), wq)


# ------------------------------------------------------------------ linear layer
@pytest.mark.parametrize("M,N,K", [(1, 4096, 1024), (2, 100, 100), (15, 77, 333), (16, 8192, 2048),
                                   (1, 1, 1), (1, 129, 8192), (3, 64, 8000), (17, 300, 1100),
                                   (32, 4096, 640), (31, 1000, 5000), (32, 20000, 128), (9, 520, 8193),
                                   (33, 512, 64), (100, 1536, 384), (1569, 1024, 1000)])
def test_linear(M, N, K):
    rs = _rs()
    x, bias, resid = draw(M, K, BF, 1), draw(1, N, BF, 2)[0], draw(M, N, BF, 3)
    w = rs.rs_fp8_quantize(draw(N, K, BF, 4, 0.0, 0.05))[0]
    a = rs.rs_fp8_quantize(x)[0]
    for kw in (dict(bias=bias, gelu=True), dict(resid=resid), dict()):
        got = rs.rs_fp8_linear(x, w, **kw)
        want, tol = epilogue_tol(a, w, kw.get("bias"), kw.get("gelu", False), kw.get("resid"), BF)
        assert ((got.double() - want).abs() <= tol).all()
    y3 = rs.rs_fp8_linear(x.view(1, M, K), w)
    assert y3.shape == (1, M, N) and torch.equal(y3[0], rs.rs_fp8_linear(x, w))
    xs = draw(M, K + 5, BF, 7)[:, 2:2 + K]
    assert torch.equal(rs.rs_fp8_linear(xs, w), rs.rs_fp8_linear(xs.contiguous(), w))


@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (2, 81, 200), (129, 130, 131), (395, 776, 200),
                                   (1000, 384, 1536)])
@pytest.mark.parametrize("dw_dtype", [BF, FP], ids=["bf16", "fp32"])
def test_linear_backward(M, N, K, dw_dtype):
    rs = _rs()
    x, w = draw(M, K, BF, 1), draw(N, K, BF, 2, 0.0, 0.05)
    dy = draw(M, N, BF, 3, 0.0, 1e-3)
    xt, wt = rs.rs_fp8_quantize(x, False, True)[1], rs.rs_fp8_quantize(w, False, True)[1]
    dx, dw, db = rs.rs_fp8_linear_backward(dy, xt, wt, bias=True, dw_dtype=dw_dtype)
    q, qt = R.quantized(dy.double()), R.quantized(dy.double().t().contiguous())
    for got, a, b, dt in ((dx, q, R.stored(wt), BF), (dw, qt, R.stored(xt), dw_dtype)):
        want, d = a @ b.T, R.product_error(a, b)
        tol = d + R.HALF_STEP[dt] * (want.abs() + d) + R.tiny(dt)
        assert ((got.double() - want).abs() <= tol).all()
    tol = (M / 64 + 40) * U * dy.double().abs().sum(0)
    assert ((db.double() - dy.double().sum(0)).abs() <= tol).all()
    only = rs.rs_fp8_linear_backward(dy, None, wt)
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None
    only = rs.rs_fp8_linear_backward(dy, xt, None, bias=True, dw_dtype=dw_dtype)
    assert only[0] is None and torch.equal(only[1], dw) and torch.equal(only[2], db)


def test_linear_backward_against_differences():
    """With the operands' stored values the layer is bilinear: its differences are exact, and
    the gradients agree with them up to the gradients' own rounding."""
    rs = _rs()
    M, N, K = 37, 50, 70
    x, w = draw(M, K, BF, 1), draw(N, K, BF, 2, 0.0, 0.05)
    dy = draw(M, N, BF, 3, 0.0, 1.0)
    xt, wt = rs.rs_fp8_quantize(x, False, True)[1], rs.rs_fp8_quantize(w, False, True)[1]
    dx, dw, _ = rs.rs_fp8_linear_backward(dy, xt, wt, dw_dtype=FP)
    q, qt = R.quantized(dy.double()), R.quantized(dy.double().t().contiguous()).T
    xv, wv = R.stored(xt).T, R.stored(wt).T
    g = torch.Generator().manual_seed(4)
    for _ in range(4):
        v = torch.randn(M, K, generator=g, dtype=R.F64).to(dev)
        n = ((xv + v) @ wv.T * q).sum() - (xv @ wv.T * q).sum()
        assert abs(n - (dx.double() * v).sum()) <= 2.0 ** -8 * (dx.double() * v).abs().sum() + 1e-6
        v = torch.randn(N, K, generator=g, dtype=R.F64).to(dev)
        n = (xv @ (wv + v).T * qt).sum() - (xv @ wv.T * qt).sum()
        assert abs(n - (dw.double() * v).sum()) <= 1e-5 * (dw.double() * v).abs().sum() + 1e-6


def test_no_rows():
    rs = _rs()
    w = draw(24, 64, BF, 2)
    wq, wt, _ = rs.rs_fp8_quantize(w, True, True)
    x = torch.empty(0, 64, dtype=BF, device=dev)
    assert rs.rs_fp8_linear(x, wq).shape == (0, 24)
    xq, xt, cs = rs.rs_fp8_quantize(x, True, True, True)
    assert (cs == 0).all()
    dx, dw, db = rs.rs_fp8_linear_backward(torch.empty(0, 24, dtype=BF, device=dev), xt, wt, bias=True)
    assert dx.shape == (0, 64) and (dw == 0).all() and dw.shape == (24, 64) and (db == 0).all()


# ------------------------------------------------------------------ the MLP
def mlp_weights(C, H, seed):
    rs = _rs()
    w1, w2 = draw(H, C, BF, seed, 0.0, 0.03), draw(C, H, BF, seed + 1, 0.0, 0.03)
    b1, b2 = draw(1, H, BF, seed + 2, 0.0, 0.1)[0], draw(1, C, BF, seed + 3, 0.0, 0.1)[0]
    return rs.rs_fp8_quantize(w1)[0], b1, rs.rs_fp8_quantize(w2)[0], b2


def mlp_expected(x, w1, b1, w2, b2, gamma, beta):
    """(expected, tolerance): errors of each stage carried into the next, a quantised value
    allowed its other neighbour only where the error reaches a border."""
    u, _, rstd, xh = R.layer_norm(x, gamma, beta, 1e-6)
    d = gamma.double().abs() * xh_error(x, rstd, xh) + 4 * U * u.abs()
    du, uq = near_border(u, d), R.quantized(u)
    v1, v2 = R.stored(w1), R.stored(w2)
    z = uq @ v1.T + b1.double()
    dz = du @ v1.abs().T + R.product_error(uq.abs() + du, v1) + U * z.abs()
    a = R.gelu(z)
    da = R.GELU_SLOPE * dz + R.GELU_ERR
    dq, aq = near_border(a, da), R.quantized(a)
    y = x.double() + aq @ v2.T + b2.double()
    dy = dq @ v2.abs().T + R.product_error(aq.abs() + dq, v2) + 3 * U * (y.abs() + x.double().abs())
    return y, dy + R.HALF_STEP[BF] * (y.abs() + dy)


@pytest.mark.parametrize("M,C,H", [(1, 64, 64), (5, 192, 768), (394, 192, 768), (130, 384, 1536),
                                   (300, 576, 2944), (200, 1024, 4096), (17, 2048, 1088)])
def test_mlp(M, C, H):
    rs = _rs()
    x = draw(M, C, BF, M + C)
    w1, b1, w2, b2 = mlp_weights(C, H, 5)
    gamma, beta = params(C, BF, 6)
    got = rs.rs_mlp_forward_fp8(x, w1, b1, w2, b2, gamma, beta)
    want, tol = mlp_expected(x, w1, b1, w2, b2, gamma, beta)
    assert ((got.double() - want).abs() <= tol).all()
    # not by the tolerance's width alone: flips at borders are few
    assert (got.double() - want).norm() <= 3e-3 * want.norm()
    ip = x.clone()
    rs.rs_mlp_forward_fp8(ip, w1, b1, w2, b2, gamma, beta, out=ip)
    assert torch.equal(ip, got)
    assert rs.rs_get_last_device_error() == 0


def test_mlp_is_its_parts():
    rs = _rs()
    x = draw(300, 384, BF, 1)
    w1, b1, w2, b2 = mlp_weights(384, 1536, 2)
    gamma, beta = params(384, BF, 3)
    u = rs.rs_ln_quantize(x, gamma, beta)
    a = rs.rs_fp8_gemm(u, w1, bias=b1, gelu=True, out_dtype=E4)
    y = rs.rs_fp8_gemm(a, w2, bias=b2, resid=x)
    assert torch.equal(y, rs.rs_mlp_forward_fp8(x, w1, b1, w2, b2, gamma, beta))


def test_training_step_of_norm_and_linear():
    """A step through norm and projection as a program runs it: each result against the
    definition applied to what the step before it produced."""
    rs = _rs()
    M, C, N = 394, 192, 776
    x, w = draw(M, C, BF, 1), draw(N, C, BF, 2, 0.0, 0.05)
    gamma, beta = params(C, FP, 3)
    bias = draw(1, N, BF, 4)[0]
    u, stats = rs.rs_ln_forward(x, gamma, beta)
    uq, ut, _ = rs.rs_fp8_quantize(u, True, True)
    wq, wt, _ = rs.rs_fp8_quantize(w, True, True)
    y = rs.rs_fp8_gemm(uq, wq, bias=bias)
    want, tol = epilogue_tol(uq, wq, bias, False, None, BF)
    assert ((y.double() - want).abs() <= tol).all()
    dy = y * 1e-3
    du, dw, db = rs.rs_fp8_linear_backward(dy, ut, wt, bias=True)
    a, b = R.quantized(dy.double()), R.stored(wt)
    want, d = a @ b.T, R.product_error(a, b)
    assert ((du.double() - want).abs() <= d + 2.0 ** -8 * (want.abs() + d)).all()
    dx, dg, dbeta = rs.rs_ln_backward(du, x, stats, gamma, dres=x)
    want, wg, wb = R.layer_norm_grad(du, x, gamma, 1e-6, x)
    assert (dx.double() - want).norm() <= 2.0 ** -8 * want.norm()
    assert (dg.double() - wg).norm() <= 1e-5 * wg.norm() and (dbeta.double() - wb).norm() <= 1e-5 * wb.norm()
    # and the whole against the unquantised layer: two e4m3 operands of 2^-4 relative rounding
    full = torch.nn.functional.linear(R.layer_norm(x, gamma, beta, 1e-6)[0], w.double(), bias.double())
    assert (y.double() - full).norm() <= 2 * 2.0 ** -4 * full.norm()


# ------------------------------------------------------------------ streams and graphs
def test_two_graphs_replay_at_once_and_streams():
    rs = _rs()
    M, C, H = 300, 384, 1536
    w1, b1, w2, b2 = mlp_weights(C, H, 2)
    gamma, beta = params(C, BF, 3)
    xs = [draw(M, C, BF, k) for k in (1, 2)]
    dys = [draw(M, C, BF, k, 0.0) for k in (3, 4)]

    def step(x, dy):
        y = rs.rs_mlp_forward_fp8(x, w1, b1, w2, b2, gamma, beta)
        u, stats = rs.rs_ln_forward(y, gamma, beta)
        z = rs.rs_fp8_linear(u, w1, bias=b1, gelu=True)
        return (y, z) + rs.rs_ln_backward(dy, y, stats, gamma, dres=u)

    want = [[t.clone() for t in step(x, dy)] for x, dy in zip(xs, dys)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, outs = [], []
    for s, x, dy in zip(streams, xs, dys):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(step(x, dy))
        graphs.append(g)
    for _ in range(5):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(p, q) for p, q in zip(o, w))
    # eager calls on two streams at once
    outs = []
    for _ in range(3):
        for s, x, dy in zip(streams, xs, dys):
            with torch.cuda.stream(s):
                outs.append(step(x, dy))
    torch.cuda.synchronize()
    for k, o in enumerate(outs):
        assert all(torch.equal(p, q) for p, q in zip(o, want[k % 2]))
    # replay with new inputs
    xs[0].copy_(xs[1])
    dys[0].copy_(dys[1])
    graphs[0].replay()
    torch.cuda.synchronize()
    graph_out = step(xs[1], dys[1])
    assert all(torch.equal(p, q) for p, q in zip(graph_out, want[1]))
    assert rs.rs_get_last_device_error() == 0


def test_scratch_belongs_to_the_stream_of_the_call():
    """With an explicit stream, scratch released on return is not handed to work on the current
    stream while the call still runs."""
    rs = _rs()
    M, C, H = 6000, 512, 2048
    w1, b1, w2, b2 = mlp_weights(C, H, 2)
    gamma, beta = params(C, BF, 3)
    x = draw(M, C, BF, 1)
    want = rs.rs_mlp_forward_fp8(x, w1, b1, w2, b2, gamma, beta)
    dy = draw(M, C, BF, 2, 0.0)
    u, stats = rs.rs_ln_forward(x, gamma, beta)
    wg = rs.rs_ln_backward(dy, x, stats, gamma)
    n = rs.rs._ws_size("rs_mlp_forward_fp8_ws_bytes", M, C, H)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs, grads = [], []
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)                 # the calls queue up behind this
    for _ in range(6):
        outs.append(rs.rs_mlp_forward_fp8(x, w1, b1, w2, b2, gamma, beta, stream=s))
        grads.append(rs.rs_ln_backward(dy, x, stats, gamma, stream=s))
        junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device=dev),
                torch.full((n // 16,), 0x7F, dtype=torch.uint8, device=dev)]
        del junk
    torch.cuda.synchronize()
    for o, g in zip(outs, grads):
        assert torch.equal(o, want) and all(torch.equal(p, q) for p, q in zip(g, wg))


def test_offsets_past_32_bits():
    """Tensors of more than 2^32 bytes and 2^31 elements: the last rows against the same rows on
    their own."""
    rs = _rs()
    M, C = (1 << 20) + 77, 2080
    x = torch.empty(M, C, dtype=BF, device=dev)
    x[:64].copy_(draw(64, C, BF, 1))
    x[64:] = x[:64].repeat((M - 64) // 64 + 1, 1)[: M - 64]
    tail = x[-100:].clone()
    gamma, beta = params(C, BF, 2)
    y, stats = rs.rs_ln_forward(x, gamma, beta)
    want, ws = rs.rs_ln_forward(tail, gamma, beta)
    assert torch.equal(y[-100:], want) and torch.equal(stats[-100:], ws)
    dx, _, db = rs.rs_ln_backward(y, x, stats, gamma)
    assert torch.equal(dx[-100:], rs.rs_ln_backward(want, tail, ws, gamma)[0])
    del y, dx
    w = rs.rs_fp8_quantize(draw(136, C, BF, 3, 0.0, 0.05))[0]
    z = rs.rs_fp8_linear(x, w)
    assert torch.equal(z[-100:], rs.rs_fp8_linear(tail, w))
    q, qt, _ = rs.rs_fp8_quantize(x, True, True)
    p = rs.rs_fp8_quantize(tail)[0]
    assert torch.equal(q.q[-100:].view(torch.uint8), p.q.view(torch.uint8))
    last = R.quantized(x[M // 128 * 128:, -8:].double().t().contiguous())
    at = R.scale_index(C, M)[-8:, -1].to(dev)
    got = qt.q[-8:, M // 128 * 128:M].double() * torch.exp2(qt.scales[at].double() - 127)[:, None]
    assert same(got, last)
    assert rs.rs_get_last_device_error() == 0


@pytest.mark.parametrize("M,N,K,skip", [(100, 128, 1024, 3), (300, 20000, 512, 0), (2000, 2048, 2048, 9)],
                         ids=["128x128", "single", "pair"])
@pytest.mark.parametrize("dtype", [BF, E4], ids=["bf16", "e4m3"])
def test_a_withheld_load_times_out_and_the_next_call_is_right(M, N, K, skip, dtype):
    rs = _rs()
    a, b = operands(M, N, K, 3)
    want = rs.rs_fp8_gemm(a, b, out_dtype=dtype)
    out = rs.rs.Fp8(want.q.clone(), want.scales.clone(), M, N) if dtype == E4 else want.clone()
    assert rs.rs_get_last_device_error() == 0
    rs.rs_debug_fp8_skip_load(a, b, out, skip, 2000)
    assert rs.rs_get_last_device_error() == rs.rs.RS_ERR_DEVICE_TIMEOUT
    assert rs.rs_get_last_device_error() == 0
    got = rs.rs_fp8_gemm(a, b, out_dtype=dtype)
    if dtype == E4:
        assert torch.equal(R.stored(got), R.stored(want))
    else:
        assert torch.equal(got, want)
    assert rs.rs_get_last_device_error() == 0


def test_refusals():
    rs = _rs()
    a, b = operands(4, 24, 64, 1)
    c = rs.rs_fp8_quantize(draw(24, 72, BF, 1))[0]
    with pytest.raises(ValueError):
        rs.rs_fp8_gemm(a, c)
    with pytest.raises(ValueError):
        rs.rs_fp8_gemm(a, b, out_dtype=HF)
    with pytest.raises(ValueError):
        rs.rs_fp8_gemm(a, b, bias=torch.zeros(23, dtype=BF, device=dev))
    with pytest.raises(ValueError):
        rs.rs_fp8_gemm(a, b, resid=torch.zeros(4, 24, device=dev))
    with pytest.raises(ValueError):
        rs.rs_fp8_gemm(a, rs.Fp8(b.q, b.scales[:100], 24, 64))
    with pytest.raises(ValueError):
        rs.rs_fp8_gemm(a, rs.Fp8(b.q, b.scales, 24, 65))
    with pytest.raises(ValueError):
        rs.rs_fp8_linear(torch.zeros(4, 64, device=dev), b)
    with pytest.raises(ValueError):
        rs.rs_fp8_linear(torch.zeros(4, 65, dtype=BF, device=dev), b)
    with pytest.raises(ValueError):
        rs.rs_fp8_linear(torch.zeros(4, 64, dtype=BF), b)
    with pytest.raises(ValueError):
        rs.rs_fp8_quantize(torch.zeros(4, 64, device=dev), colsum=True)
    with pytest.raises(rs.RsError):
        rs.rs_fp8_linear(torch.zeros(40, 64, dtype=BF, device=dev), b,
                         ws=torch.empty(256, dtype=torch.uint8, device=dev))
    assert rs.rs_get_last_device_error() == 0
