"""The layer norm and its gradients where each row of threads walks more rows than its ring in
shared memory holds, with rows that change their place against 16 bytes (needs a B200). Tolerances
as in test_norm_gpu.py."""
import pytest
import torch

from test_norm_gpu import BF, FP, HF, check_bwd, check_fwd, dev, draw, params

pytestmark = pytest.mark.gpu

# rows of a row of threads: at least 8 forward (4 in its ring) and 16 backward (3 in its ring)
SHAPES = [(20001, 1001), (60000, 77), (40001, 333), (40001, 334)]


def _rs():
    import free_vit_token_b200 as rs
    return rs


@pytest.mark.parametrize("dtype", [BF, HF, FP], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,C", SHAPES)
def test_forward(M, C, dtype):
    rs = _rs()
    x = draw(M, C, dtype, M + C)
    gamma, beta = params(C, dtype, C)
    y, stats = rs.rs_ln_forward(x, gamma, beta)
    check_fwd(x, gamma, beta, y, stats)
    # strided and in place: the same values
    buf = torch.full((M, C + 5), 7.0, dtype=dtype, device=dev)
    v = buf[:, 3:3 + C]
    v.copy_(x)
    rs.rs_ln_forward(v, gamma, beta, y=v)
    assert torch.equal(v, y)
    assert (buf[:, :3] == 7).all() and (buf[:, 3 + C:] == 7).all()


@pytest.mark.parametrize("dtype", [BF, HF, FP], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,C", SHAPES)
def test_backward(M, C, dtype):
    rs = _rs()
    x, dy, dres = draw(M, C, dtype, 1), draw(M, C, dtype, 2, 0.0), draw(M, C, dtype, 3, 0.0)
    gamma, _ = params(C, dtype, 4)
    _, stats = rs.rs_ln_forward(x)
    got = rs.rs_ln_backward(dy, x, stats, gamma, dres)
    check_bwd(dy, x, gamma, dres, got)
    # strided and in place, each tensor with an offset of its own
    buf = torch.full((M, C + 7), 7.0, dtype=dtype, device=dev)
    v = buf[:, 5:5 + C]
    v.copy_(dres)
    xs = torch.empty(M, C + 3, dtype=dtype, device=dev)[:, 1:1 + C]
    xs.copy_(x)
    again = rs.rs_ln_backward(dy, xs, stats, gamma, v, dx=v)
    assert all(torch.equal(p, q) for p, q in zip(again, got))
    assert (buf[:, :5] == 7).all() and (buf[:, 5 + C:] == 7).all()


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_wide_rows(dtype):
    """One row of threads per block, several rows each."""
    rs = _rs()
    M, C = 1700, 5003
    x, dy = draw(M, C, dtype, 1), draw(M, C, dtype, 2, 0.0)
    gamma, beta = params(C, dtype, 3)
    y, stats = rs.rs_ln_forward(x, gamma, beta)
    check_fwd(x, gamma, beta, y, stats)
    check_bwd(dy, x, gamma, None, rs.rs_ln_backward(dy, x, stats, gamma))
