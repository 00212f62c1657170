"""rs_fp8_linear on a few rows beside other work (needs a B200)."""
import pytest
import torch

from test_norm_gpu import draw, params

pytestmark = pytest.mark.gpu
dev = torch.device("cuda:0")
BF = torch.bfloat16


def _rs():
    import free_vit_token_b200 as rs
    return rs


def test_beside_cta_pairs_of_another_stream():
    """The bf16 products of 64-column tiles (CTA pairs that take an SM's whole tensor memory and
    leave shared memory for a CTA of this kernel) on one stream, few-row clusters on another:
    none holds tensor memory while it waits for its cluster, so both get through, with the
    results that each has alone."""
    rs = _rs()
    C = H = 1088
    x = draw(2000, C, BF, 1)
    W1, W2 = draw(H, C, BF, 2, 0.0, 0.03), draw(C, H, BF, 3, 0.0, 0.03)
    b1, b2 = draw(1, H, BF, 4)[0], draw(1, C, BF, 5)[0]
    gamma, beta = params(C, BF, 6)
    want = rs.rs_mlp_forward(x, W1, b1, W2, b2, gamma, beta)
    few = []
    for M, N, K in ((8, 1024, 256), (1, 4096, 512), (16, 2048, 384)):
        v, w = draw(M, K, BF, M), rs.rs_fp8_quantize(draw(N, K, BF, N, 0.0, 0.05))[0]
        few.append((v, w, rs.rs_fp8_linear(v, w)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    big, small = [], []
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            big.append(rs.rs_mlp_forward(x, W1, b1, W2, b2, gamma, beta))
        with torch.cuda.stream(streams[1]):
            for _ in range(4):
                small.extend((rs.rs_fp8_linear(v, w), y) for v, w, y in few)
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in big)
    assert all(torch.equal(y, z) for y, z in small)
    assert rs.rs_get_last_device_error() == 0


# a cluster of several CTAs, one CTA a reduction, up to 32 rows
@pytest.mark.parametrize("M,N,K", [(8, 1000, 2048), (16, 300, 128), (20, 4096, 640)])
def test_a_withheld_weight_tile_times_out_and_the_next_call_is_right(M, N, K):
    rs = _rs()
    x, w = draw(M, K, BF, 1), rs.rs_fp8_quantize(draw(N, K, BF, 2, 0.0, 0.05))[0]
    want = rs.rs_fp8_linear(x, w)
    out = want.clone()
    assert rs.rs_get_last_device_error() == 0
    rs.rs_debug_fp8_linear_skip_load(x, w, out, 2000)
    assert rs.rs_get_last_device_error() == rs.rs.RS_ERR_DEVICE_TIMEOUT
    assert rs.rs_get_last_device_error() == 0
    assert torch.equal(rs.rs_fp8_linear(x, w), want)
    assert rs.rs_get_last_device_error() == 0
