"""Host-side checks of the layer norm and 8-bit entry points: what they refuse, before
anything is launched (no GPU)."""
import pytest

import free_vit_token_b200.rs as rs

F = 0x100000   # aligned fake device address, never dereferenced on these paths
BF, HF, FP, E4 = rs.RS_BF16, rs.RS_FP16, rs.RS_FP32, rs.RS_E4M3
OK, NULL, SHAPE, ALIGN, NOMEM = (rs.RS_OK, rs.RS_ERR_NULL, rs.RS_ERR_SHAPE, rs.RS_ERR_ALIGN,
                                 rs.RS_ERR_NO_MEM)
BIG = 1 << 40


def fwd(x=F, ldx=64, M=4, C=64, dt=BF, g=F, b=F, pdt=BF, eps=1e-6, y=F, ldy=64, st=F):
    return rs.lib().rs_ln_forward(x, ldx, M, C, dt, g, b, pdt, eps, y, ldy, st, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=0), OK), (dict(M=0, x=None, y=None), OK), (dict(M=-1), SHAPE), (dict(M=1 << 27), SHAPE),
    (dict(C=0, ldx=0), SHAPE), (dict(C=8193, ldx=8193, ldy=8193), SHAPE), (dict(dt=E4), SHAPE),
    (dict(dt=-1), SHAPE), (dict(pdt=HF), SHAPE), (dict(dt=FP, pdt=BF), SHAPE), (dict(ldx=63), SHAPE),
    (dict(ldy=63), SHAPE), (dict(eps=0.0), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(x=None), NULL), (dict(y=None), NULL), (dict(x=F + 1), ALIGN), (dict(y=F + 1), ALIGN),
    (dict(g=F + 1), ALIGN), (dict(st=F + 4), ALIGN), (dict(pdt=FP, g=F + 2), ALIGN)])
def test_ln_forward(kw, want):
    assert fwd(**kw) == want


def lnq(x=F, ldx=64, M=4, C=64, dt=BF, g=F, pdt=BF, q=F, ldq=64, s=F, st=None):
    return rs.lib().rs_ln_quantize(x, ldx, M, C, dt, g, F, pdt, 1e-6, q, ldq, s, st, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=0), OK), (dict(dt=FP, pdt=FP), SHAPE), (dict(C=60), SHAPE), (dict(ldq=56), SHAPE),
    (dict(ldq=72), SHAPE), (dict(q=None), NULL), (dict(s=None), NULL), (dict(q=F + 8), ALIGN),
    (dict(s=F + 8), ALIGN), (dict(x=F + 8), ALIGN), (dict(ldx=68), ALIGN), (dict(g=F + 2), ALIGN)])
def test_ln_quantize(kw, want):
    assert lnq(**kw) == want


def bwd(dy=F, ldy=64, x=F, ldx=64, dr=F, ldr=64, st=F, g=F, pdt=BF, M=4, C=64, dt=BF, dx=F, lddx=64,
        dg=F, db=F, ws=F, n=BIG):
    return rs.lib().rs_ln_backward(dy, ldy, x, ldx, dr, ldr, st, g, pdt, M, C, dt, dx, lddx, dg, db,
                                   ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dx=None, dg=None, db=None), OK), (dict(M=0, dg=None, db=None), OK), (dict(M=-1), SHAPE),
    (dict(dt=E4), SHAPE), (dict(pdt=HF), SHAPE), (dict(ldy=63), SHAPE), (dict(ldr=63), SHAPE),
    (dict(lddx=63), SHAPE), (dict(dy=None), NULL), (dict(x=None), NULL), (dict(st=None), NULL),
    (dict(dy=F + 1), ALIGN), (dict(dx=F + 1), ALIGN), (dict(st=F + 4), ALIGN), (dict(dg=F + 2), ALIGN)])
def test_ln_backward(kw, want):
    assert bwd(**kw) == want


def quant(x=F, ldx=200, R=4, K=200, dt=BF, q=F, ldq=208, s=F, qt=F, ldqt=16, st=F, cs=F, ws=F, n=BIG):
    return rs.lib().rs_fp8_quantize(x, ldx, R, K, dt, q, ldq, s, qt, ldqt, st, cs, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(R=0, cs=None), OK), (dict(q=None, qt=None, cs=None), OK), (dict(R=-1), SHAPE),
    (dict(K=0), SHAPE), (dict(dt=E4), SHAPE), (dict(ldx=199), SHAPE), (dict(ldq=200), SHAPE),
    (dict(ldq=192), SHAPE), (dict(ldqt=0), SHAPE), (dict(ldqt=20), SHAPE), (dict(x=None), NULL),
    (dict(s=None), NULL), (dict(st=None), NULL), (dict(qt=None), NULL), (dict(ws=None), NULL),
    (dict(x=F + 1), ALIGN), (dict(q=F + 8), ALIGN), (dict(qt=F + 8), ALIGN), (dict(ws=F + 16), ALIGN),
    (dict(n=64), NOMEM)])
def test_quantize(kw, want):
    assert quant(**kw) == want


def gemm(a=F, lda=208, sa=F, b=F, ldb=208, sb=F, M=4, N=24, K=200, bias=F, gelu=0, r=None, ldr=24,
         o=F, ldo=24, dt=BF, so=None):
    return rs.lib().rs_fp8_gemm(a, lda, sa, b, ldb, sb, M, N, K, bias, gelu, r, ldr, o, ldo, dt, so,
                                None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=0), OK), (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(K=0), SHAPE),
    (dict(M=1 << 26, N=1 << 26, ldo=1 << 26), SHAPE), (dict(dt=HF), SHAPE), (dict(gelu=2), SHAPE),
    (dict(ldo=23), SHAPE), (dict(r=F, ldr=23), SHAPE), (dict(lda=200), SHAPE), (dict(ldb=192), SHAPE),
    (dict(so=F), SHAPE), (dict(dt=E4, so=F, r=F), SHAPE), (dict(dt=E4, so=F, ldo=24), SHAPE),
    (dict(a=None), NULL), (dict(sb=None), NULL), (dict(o=None), NULL), (dict(dt=E4, ldo=32), NULL),
    (dict(a=F + 8), ALIGN), (dict(bias=F + 2), ALIGN), (dict(o=F + 1), ALIGN),
    (dict(dt=FP, o=F + 2), ALIGN), (dict(r=F + 1), ALIGN)])
def test_gemm(kw, want):
    assert gemm(**kw) == want


@pytest.mark.parametrize("skip,us,want", [(-1, 100, SHAPE), (2, 100, SHAPE), (0, 0, SHAPE),
                                          (0, 10000001, SHAPE), (1, 100, NULL)])
def test_debug_skip_load(skip, us, want):
    assert rs.lib().rs_debug_fp8_skip_load(None, 208, F, F, 208, F, 4, 24, 200, F, 24, BF, None, skip, us,
                                           None) == want


def linear(x=F, ldx=200, M=40, K=200, N=24, w=F, ldw=208, sw=F, bias=F, gelu=0, r=None, ldr=24, o=F,
           ldo=24, ws=F, n=BIG):
    return rs.lib().rs_fp8_linear(x, ldx, M, K, N, w, ldw, sw, bias, gelu, r, ldr, o, ldo, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=0), OK), (dict(K=0), SHAPE), (dict(ldx=199), SHAPE), (dict(ldo=23), SHAPE),
    (dict(ldw=200), SHAPE), (dict(x=None), NULL), (dict(w=None), NULL), (dict(o=None), NULL),
    (dict(ws=None), NULL), (dict(ws=F + 128), ALIGN), (dict(n=100), NOMEM), (dict(x=F + 1), ALIGN)])
def test_linear(kw, want):
    assert linear(**kw) == want


def lbwd(dy=F, ldy=24, M=4, N=24, K=200, xt=F, ldxt=16, sx=F, wt=F, ldwt=32, sw=F, dx=F, lddx=200,
         dw=F, lddw=200, dt=BF, db=F, ws=F, n=BIG):
    return rs.lib().rs_fp8_linear_backward(dy, ldy, M, N, K, xt, ldxt, sx, wt, ldwt, sw, dx, lddx, dw,
                                           lddw, dt, db, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dx=None, dw=None, db=None), OK), (dict(M=0, dw=None, db=None), OK), (dict(N=0), SHAPE),
    (dict(dt=HF), SHAPE), (dict(ldy=23), SHAPE), (dict(lddx=199), SHAPE), (dict(lddw=199), SHAPE),
    (dict(ldxt=8), SHAPE), (dict(ldwt=16), SHAPE), (dict(dy=None), NULL), (dict(xt=None), NULL),
    (dict(sw=None), NULL), (dict(ws=None), NULL), (dict(n=100), NOMEM), (dict(dy=F + 1), ALIGN)])
def test_linear_backward(kw, want):
    assert lbwd(**kw) == want


def mlp(x=F, M=4, C=64, H=128, w1=F, ld1=64, s1=F, b1=F, w2=F, ld2=128, s2=F, y=F, ws=F, n=BIG):
    return rs.lib().rs_mlp_forward_fp8(x, M, C, H, w1, ld1, s1, b1, w2, ld2, s2, F, F, F, y, ws, n,
                                       None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=0), OK), (dict(C=100), SHAPE), (dict(H=100), SHAPE), (dict(M=-1), SHAPE),
    (dict(ld1=48), SHAPE), (dict(x=None), NULL), (dict(y=None), NULL), (dict(b1=None), NULL),
    (dict(s2=None), NULL), (dict(x=F + 8), ALIGN), (dict(y=F + 8), ALIGN), (dict(ws=None), NULL),
    (dict(n=100), NOMEM)])
def test_mlp_forward_fp8(kw, want):
    assert mlp(**kw) == want


def test_sizes():
    L = rs.lib()
    assert L.rs_fp8_scale_bytes(1, 1) == 512 and L.rs_fp8_scale_bytes(129, 513) == 2048
    assert L.rs_fp8_scale_bytes(0, 64) == 0 and L.rs_fp8_scale_bytes(4, 0) == 0
    assert L.rs_fp8_linear_ws_bytes(33, 200) >= 33 * 208 + 512
    assert L.rs_fp8_linear_ws_bytes(16, 8192) == 0 and L.rs_fp8_linear_ws_bytes(16, 8193) > 0
    assert L.rs_fp8_linear_ws_bytes(17, 8192) > 0
    assert L.rs_fp8_quantize_ws_bytes(129, 200) >= 2 * 200 * 4
    assert L.rs_fp8_linear_backward_ws_bytes(130, 24) >= 130 * 32 + 24 * 144 + 2 * 24 * 4
    assert L.rs_mlp_forward_fp8_ws_bytes(10, 64, 128) >= 10 * 192
    assert L.rs_mlp_forward_fp8_ws_bytes(10, 65, 128) == 0
    # sizes past 32 bits do not wrap
    assert L.rs_fp8_scale_bytes((1 << 27) - 1, 8192) == (1 << 20) * 16 * 512
    assert L.rs_fp8_linear_ws_bytes((1 << 27) - 1, 4096) > 1 << 38


def test_python_refusals_need_no_gpu():
    import torch

    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    cpu = x.get_device()
    with pytest.raises(ValueError, match="CUDA device"):
        rs._device(x, "x")
    with pytest.raises(ValueError, match="CUDA device"):
        rs._rows(x, "x", 0)
    with pytest.raises(ValueError, match="contiguous"):
        rs._rows(x.t(), "x", cpu)
    with pytest.raises(ValueError, match="rows overlap"):
        rs._rows(x.as_strided((2, 64), (32, 1)), "x", cpu)
    with pytest.raises(ValueError, match="wanted"):
        rs._rows(x, "x", cpu, torch.float32)
    with pytest.raises(ValueError, match="rows of 63"):
        rs._rows(x, "x", cpu, width=63)
    with pytest.raises(ValueError, match="matrix"):
        rs._rows(x.view(2, 2, 64)[:, :, :32], "x", cpu)
    assert rs._rows(x[:, 8:40], "x", cpu)[1:] == (64, 4)
    assert rs._rows(x[:1, 8:40], "x", cpu)[1] >= 32
    with pytest.raises(ValueError):
        rs._float_type(torch.zeros(2, dtype=torch.float64))
    with pytest.raises(ValueError):
        rs._params(x, cpu, 64, torch.zeros(64, dtype=torch.float16), None)
