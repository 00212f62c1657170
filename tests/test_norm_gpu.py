"""The layer norm and its gradients against 64 bits (needs a B200).

Tolerances. A row of C values is summed by chains of at most 16 additions and 9 levels between
threads, each rounding by 2^-24 of what it holds: the mean is off by at most 27 * 2^-24 max|x|,
rstd by twice that relative to itself and a few roundings more. With xh = (x - mean) rstd,
  |d xh| <= 2^-24 (32 max|x| rstd + 80 |xh|),
and y adds half a step of its type. The gradients carry |d xh| through their formulas; sums
over rows add (rows of a thread + 24) roundings of 2^-24 of the magnitudes summed."""
import ctypes

import pytest
import torch

import fp8_ref as R

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")
U = 2.0 ** -24
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6


def _rs():
    import free_vit_token_b200 as rs
    return rs


def draw(M, C, dtype, seed, mean=0.3, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, C, generator=g) * scale + mean
    return x.to(dtype).to(dev)


def params(C, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return ((1 + 0.1 * torch.randn(C, generator=g)).to(dtype).to(dev),
            (0.1 * torch.randn(C, generator=g)).to(dtype).to(dev))


def xh_error(x, rstd, xh):
    return U * (32 * x.double().abs().amax(-1, keepdim=True) * rstd + 80 * xh.abs())


def check_fwd(x, gamma, beta, y, stats, eps=EPS):
    want, mean, rstd, xh = R.layer_norm(x, gamma, beta, eps)
    top = x.double().abs().amax(-1, keepdim=True)
    g = 1.0 if gamma is None else gamma.double().abs()
    tol = g * xh_error(x, rstd, xh) + 4 * U * want.abs()
    h = R.HALF_STEP[y.dtype]
    tol = tol + h * (want.abs() + tol) + R.tiny(y.dtype)
    assert ((y.double() - want).abs() <= tol).all()
    assert ((stats[:, :1].double() - mean).abs() <= 27 * U * top).all()
    assert ((stats[:, 1:].double() - rstd).abs() <= rstd * U * (64 * top * rstd + 80)).all()


@pytest.mark.parametrize("dtype", [BF, HF, FP], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,C", [(1, 1), (1, 8), (5, 7), (33, 64), (394, 192), (65, 256), (9, 264),
                                 (100, 500), (257, 512), (77, 768), (31, 1000), (300, 1024),
                                 (50, 1025), (17, 2048), (13, 2056), (5, 4096), (3, 4100),
                                 (4, 8191), (2, 8192), (5000, 40)])
def test_forward(M, C, dtype):
    rs = _rs()
    x = draw(M, C, dtype, M + C)
    for pd in {dtype, FP}:
        gamma, beta = params(C, pd, C)
        y, stats = rs.rs_ln_forward(x, gamma, beta, eps=EPS)
        check_fwd(x, gamma, beta, y, stats)
    y, stats = rs.rs_ln_forward(x)
    check_fwd(x, None, None, y, stats)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_forward_strided_unaligned_and_in_place(dtype):
    rs = _rs()
    M, C = 37, 200
    gamma, beta = params(C, dtype, 1)
    for off, ld in ((0, 208), (0, 203), (1, 208), (3, 201), (8, 264)):
        buf = draw(M, ld, dtype, 2)
        flat = torch.cat([torch.zeros(16, dtype=dtype, device=dev), buf.flatten()])
        x = flat[16 + off:16 + off + (M - 1) * ld + C].as_strided((M, C), (ld, 1)) if off + C <= ld \
            else None
        if x is None:
            continue
        want = x.clone()
        out = torch.full((M + 2, ld), 7.0, dtype=dtype, device=dev)
        y, stats = rs.rs_ln_forward(x, gamma, beta, y=out[1:M + 1, :C])
        check_fwd(want, gamma, beta, y, stats)
        assert (out[0] == 7).all() and (out[M + 1] == 7).all() and (out[:, C:] == 7).all()
        assert torch.equal(x, want)
        rs.rs_ln_forward(x, gamma, beta, y=x)              # in place
        assert torch.equal(x, y)


def test_forward_mean_far_from_zero_and_constant_rows():
    rs = _rs()
    x = draw(64, 1024, FP, 3, mean=1000.0)
    gamma, beta = params(1024, FP, 3)
    y, stats = rs.rs_ln_forward(x, gamma, beta)
    check_fwd(x, gamma, beta, y, stats)
    c = torch.full((3, 768), 0.625, dtype=BF, device=dev)  # the mean is exact: y = beta
    gamma, beta = params(768, BF, 4)
    y, _ = rs.rs_ln_forward(c, gamma, beta)
    assert torch.equal(y, beta.expand(3, -1))


def test_forward_nonfinite_rows_stay_apart():
    rs = _rs()
    x = draw(6, 320, FP, 5)
    x[1, 7] = float("nan")
    x[3, 0] = float("inf")
    y, stats = rs.rs_ln_forward(x)
    keep = [0, 2, 4, 5]
    check_fwd(x[keep], None, None, y[keep], stats[keep])
    assert y[1].isnan().all() and y[3].isnan().all()


def test_more_dimensions_and_no_rows():
    rs = _rs()
    x = draw(24, 192, BF, 6).view(2, 3, 4, 192)
    y, stats = rs.rs_ln_forward(x)
    assert y.shape == x.shape and stats.shape == (24, 2)
    check_fwd(x.view(24, 192), None, None, y.view(24, 192), stats)
    e = torch.empty(0, 192, dtype=BF, device=dev)
    y, stats = rs.rs_ln_forward(e)
    assert y.shape == (0, 192)
    dx, dg, db = rs.rs_ln_backward(e, e, stats)
    assert dx.shape == (0, 192) and (dg == 0).all() and (db == 0).all()


# ------------------------------------------------------------------ backward
def check_bwd(dy, x, gamma, dres, got, eps=EPS):
    dx, dg, db = got
    want, wg, wb = R.layer_norm_grad(dy, x, gamma, eps, dres)
    _, _, rstd, xh = R.layer_norm(x, None, None, eps)
    M, C = x.shape
    d = xh_error(x, rstd, xh)
    dyd = dy.double()
    w = dyd if gamma is None else dyd * gamma.double()
    aw = w.abs()
    chain = 48 * U
    m1 = chain * aw.mean(-1, keepdim=True)
    m2a = (w * xh).abs().mean(-1, keepdim=True)
    m2 = chain * m2a + (aw * d).mean(-1, keepdim=True)
    inner = U * 4 * (aw + aw.mean(-1, keepdim=True) + xh.abs() * m2a) + m1 + xh.abs() * m2 + d * m2a
    top = x.double().abs().amax(-1, keepdim=True)
    size = aw + aw.mean(-1, keepdim=True) + xh.abs() * m2a
    tol = rstd * (inner + size * U * (64 * top * rstd + 80))
    if dres is not None:
        tol = tol + U * (want.abs() + dres.double().abs())
    tol = tol + R.HALF_STEP[dx.dtype] * (want.abs() + tol) + R.tiny(dx.dtype)
    assert ((dx.double() - want).abs() <= tol).all()
    rows = M / (148 * (12 if C <= 1024 else 1)) + 12 + 24 + 20
    assert ((db.double() - wb).abs() <= rows * U * dyd.abs().sum(0)).all()
    tg = rows * U * (dyd * xh).abs().sum(0) + (dyd.abs() * d).sum(0)
    assert ((dg.double() - wg).abs() <= tg).all()


@pytest.mark.parametrize("dtype", [BF, HF, FP], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,C", [(1, 1), (1, 8), (5, 7), (33, 64), (394, 192), (65, 256), (9, 264),
                                 (257, 512), (77, 768), (31, 1001), (300, 1024), (50, 1030),
                                 (17, 2048), (13, 2056), (5, 4096), (7, 4100), (4, 8191), (2, 8192),
                                 (6000, 40), (4001, 768), (512, 192), (513, 192),
                                 (256, 1000), (300, 2000), (33, 8000)])
def test_backward(M, C, dtype):
    rs = _rs()
    x, dy, dres = draw(M, C, dtype, 1), draw(M, C, dtype, 2, 0.0), draw(M, C, dtype, 3, 0.0)
    gamma, _ = params(C, dtype, 4)
    _, stats = rs.rs_ln_forward(x, eps=EPS)
    a = rs.rs_ln_backward(dy, x, stats, gamma, dres)
    check_bwd(dy, x, gamma, dres, a)
    b = rs.rs_ln_backward(dy, x, stats, gamma, dres)
    assert all(torch.equal(p, q) for p, q in zip(a, b))       # the same bits every time
    check_bwd(dy, x, None, None, rs.rs_ln_backward(dy, x, stats))


def test_backward_against_differences():
    rs = _rs()
    M, C = 4, 24
    x, dy = draw(M, C, FP, 7), draw(M, C, FP, 8, 0.0)
    gamma, beta = params(C, FP, 9)
    _, stats = rs.rs_ln_forward(x, eps=EPS)
    dx, dg, db = rs.rs_ln_backward(dy, x, stats, gamma)
    f = lambda x_, g_, b_: float((R.layer_norm(x_, g_, b_, EPS)[0] * dy.double()).sum())  # noqa: E731
    h, xd, gd, bd = 1e-5, x.double(), gamma.double(), beta.double()
    g = torch.Generator().manual_seed(10)
    for _ in range(8):
        v = torch.randn(M, C, generator=g, dtype=torch.float64).to(dev)
        n = (f(xd + h * v, gd, bd) - f(xd - h * v, gd, bd)) / (2 * h)
        assert abs(n - float((dx.double() * v).sum())) <= 1e-4 * float((dx.double() * v).abs().sum())
        v = torch.randn(C, generator=g, dtype=torch.float64).to(dev)
        n = (f(xd, gd + h * v, bd) - f(xd, gd - h * v, bd)) / (2 * h)
        assert abs(n - float((dg.double() * v).sum())) <= 1e-4 * float((dg.double() * v).abs().sum())
        n = (f(xd, gd, bd + h * v) - f(xd, gd, bd - h * v)) / (2 * h)
        assert abs(n - float((db.double() * v).sum())) <= 1e-4 * float((db.double() * v).abs().sum())


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_backward_strided_in_place_and_parts(dtype):
    rs = _rs()
    M, C, ld = 570, 136, 147
    xs, ys, ds = (draw(M, ld, dtype, k) for k in (1, 2, 3))
    x, dy, dres = xs[:, 3:3 + C], ys[:, 1:1 + C], ds[:, 5:5 + C]
    gamma, _ = params(C, FP, 4)
    _, stats = rs.rs_ln_forward(x, eps=EPS)
    rest = ds.clone()
    want = rs.rs_ln_backward(dy, x, stats, gamma, dres)
    check_bwd(dy, x, gamma, dres.clone(), want)
    got = rs.rs_ln_backward(dy, x, stats, gamma, dres, dx=dres)     # in place
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(ds[:, :5], rest[:, :5]) and torch.equal(ds[:, 5 + C:], rest[:, 5 + C:])
    # parts: only dx (no scratch), only dbeta
    L, p = rs.lib(), lambda t: t.data_ptr()  # noqa: E731
    xc, yc = x.contiguous(), dy.contiguous()
    full = rs.rs_ln_backward(yc, xc, stats, gamma)
    dt = rs.RS_BF16 if dtype == BF else rs.RS_FP32
    dx = torch.empty_like(xc)
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert L.rs_ln_backward(p(yc), C, p(xc), C, None, 0, p(stats), p(gamma), rs.RS_FP32, M, C, dt,
                            p(dx), C, None, None, None, 0, s) == 0
    assert torch.equal(dx, full[0])
    db = torch.empty(C, device=dev)
    n = L.rs_ln_backward_ws_bytes(M, C)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    assert L.rs_ln_backward(p(yc), C, p(xc), C, None, 0, p(stats), p(gamma), rs.RS_FP32, M, C, dt,
                            None, 0, None, p(db), p(ws), n, s) == 0
    assert torch.equal(db, full[2])
    assert L.rs_ln_backward(p(yc), C, p(xc), C, None, 0, p(stats), p(gamma), rs.RS_FP32, M, C, dt,
                            None, 0, None, p(db), p(ws), n - 1, s) == rs.rs.RS_ERR_NO_MEM


# ------------------------------------------------------------------ quantised output
def near_border(y, d):
    """Where a value within d of y (64 bits) may round to another e4m3 value or its block take
    another scale: the values' possible difference from quantized(y), else zero."""
    e = R.block_exponents(y)
    f = R.spread(e, y.shape[1])
    K = y.shape[1]
    # a block whose largest value lies within d of a border may take the next scale
    pad = (-(-K // 128)) * 128
    a, b = (torch.zeros(y.shape[0], pad, dtype=torch.float64, device=y.device) for _ in range(2))
    a[:, :K] = (y.abs() - d).clamp(min=0)
    b[:, :K] = y.abs() + d
    lo = R.block_exponents(a)
    hi = R.block_exponents(torch.where(b < 1e300, b, torch.zeros_like(b)))
    moved = R.spread((lo != hi).double().log2().nan_to_num(neginf=-1000), K) > 0.5
    v = y / f
    s = R.e4m3_step(v)
    t = (v / s - torch.floor(v / s) - 0.5).abs() * s          # distance to the next tie
    flip = t <= d / f
    return torch.where(moved, 2 * s * f + d, torch.where(flip, s * f + d, torch.zeros_like(d)))


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("M,C", [(1, 8), (3, 64), (394, 192), (129, 200), (33, 512), (260, 768),
                                 (50, 1024), (20, 1160), (9, 2048), (5, 4104), (3, 8192)])
def test_quantized_output(M, C, dtype):
    rs = _rs()
    x = draw(M, C, dtype, M * C)
    gamma, beta = params(C, dtype, C)
    out = rs.rs._fp8_empty(M, C, dev)
    out.q.view(torch.uint8).fill_(0x55)
    stats = torch.empty(M, 2, device=dev)
    rs.rs_ln_quantize(x, gamma, beta, EPS, out=out, stats=stats)
    assert (out.q.view(torch.uint8)[:, C:] == 0x55).all()
    y, _, rstd, xh = R.layer_norm(x, gamma, beta, EPS)
    d = gamma.double().abs() * xh_error(x, rstd, xh) + 4 * U * y.abs()
    diff = (R.stored(out) - R.quantized(y)).abs()
    assert (diff <= near_border(y, d)).all()
    assert (diff == 0).double().mean() > 0.99
    _, want = rs.rs_ln_forward(x, gamma, beta, EPS)
    assert torch.equal(stats, want)


def test_quantized_output_nonfinite():
    rs = _rs()
    x = draw(4, 256, BF, 5)
    x[2, 200] = float("nan")
    q = rs.rs_ln_quantize(x)
    v = R.stored(q)
    assert v[2].isnan().all() and not v[[0, 1, 3]].isnan().any()


def test_refusals():
    rs = _rs()
    x = draw(4, 64, BF, 1)
    with pytest.raises(ValueError):
        rs.rs_ln_forward(x.double())
    with pytest.raises(ValueError):
        rs.rs_ln_forward(x, torch.ones(63, dtype=BF, device=dev))
    with pytest.raises(ValueError):
        rs.rs_ln_forward(x, torch.ones(64, dtype=BF, device=dev), torch.ones(64, device=dev))
    with pytest.raises(ValueError):
        rs.rs_ln_forward(x, y=torch.empty(4, 63, dtype=BF, device=dev))
    with pytest.raises(ValueError):
        rs.rs_ln_forward(x.cpu())
    with pytest.raises(rs.RsError):
        rs.rs_ln_forward(x, eps=0.0)
    with pytest.raises(rs.RsError):
        rs.rs_ln_forward(draw(2, 8200, BF, 1))
    with pytest.raises(ValueError):
        rs.rs_ln_backward(x[:3], x, torch.empty(4, 2, device=dev))
    with pytest.raises(rs.RsError):
        rs.rs_ln_quantize(draw(4, 60, BF, 1))
    with pytest.raises(rs.RsError):
        rs.rs_ln_quantize(x.float())
    assert rs.rs_get_last_device_error() == 0
