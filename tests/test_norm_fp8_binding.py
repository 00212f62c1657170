"""The Python binding of the layer norm and 8-bit calls: what it passes on and keeps (no GPU)."""
import pytest
import torch

import free_vit_token_b200.rs as rs

BF = torch.bfloat16


@pytest.mark.parametrize("shape", [((1 << 32) + 4, 0), (1 << 31, 8), (1 << 16, 1 << 16, 1),
                                   (0, (1 << 32) + 64), (0, 1 << 31), (1, (1 << 32) + 64)])
def test_sizes_past_an_int_are_refused(shape):
    """They would reach the library as what is left of them in 32 bits."""
    x = torch.empty(shape, dtype=BF, device="meta")  # a shape without memory
    with pytest.raises(ValueError, match="2\\^31"):
        rs._rows(x, "x", x.get_device())


def test_sizes_within_an_int_pass():
    x = torch.empty((1 << 31) - 1, 0, dtype=BF)
    assert rs._rows(x, "x", x.get_device())[2] == (1 << 31) - 1
    assert rs._rows(torch.empty(0, (1 << 31) - 1, dtype=BF), "x", x.get_device())[1] == (1 << 31) - 1


def test_scale_bytes_of_sizes_past_an_int():
    assert rs.rs_fp8_scale_bytes(4, 64) == 512
    for rows, K in (((1 << 32) + 4, 64), (4, (1 << 32) + 64), (-(1 << 32) + 4, 64)):
        assert rs.rs_fp8_scale_bytes(rows, K) == 0


def test_operand_with_a_negative_width():
    q = torch.empty(4, 64, dtype=torch.float8_e4m3fn)
    t = rs.Fp8(q, torch.empty(512, dtype=torch.uint8), 4, -(1 << 32) + 64)
    with pytest.raises(ValueError, match="shorter than K"):
        rs._fp8(t, "w", q.get_device())


class _Sizes:
    """A library whose layer norm needs scratch past 1000 rows: by device, none while it cannot
    ask the device."""

    def __init__(self):
        self.sms, self.asked = 0, 0

    def rs_ln_backward_ws_bytes(self, M, C):
        self.asked += 1
        return self.sms * 100 if M > 1000 else 0


@pytest.fixture
def sizes(monkeypatch):
    lib = _Sizes()
    monkeypatch.setattr(rs, "lib", lambda: lib)
    monkeypatch.setattr(rs, "_ws_sizes", {}, raising=False)

    def ask(dev, M, sms):
        lib.sms = sms
        return rs._ws(None, torch.device("cpu"), dev, "rs_ln_backward_ws_bytes", M, 333)[1]
    return lib, ask


def test_scratch_sizes_are_kept_by_device(sizes):
    """What one device answered is not another's size."""
    lib, ask = sizes
    assert [ask(0, 7001, 10), ask(1, 7001, 20), ask(0, 7001, 10)] == [1000, 2000, 1000]
    assert lib.asked == 2


def test_a_failed_size_query_is_not_kept(sizes):
    lib, ask = sizes
    assert [ask(0, 7003, 0), ask(0, 7003, 30), ask(0, 7003, 30)] == [0, 3000, 3000]


def test_no_scratch_is_kept_too(sizes):
    lib, ask = sizes
    assert ask(0, 12, 10) == 0
    n = lib.asked
    assert ask(0, 12, 10) == 0 and lib.asked == n


@pytest.mark.parametrize("M,N,K,us", [(0, 64, 64, 100), (33, 64, 64, 100), (17, 8193, 64, 100), (4, 64, 8193, 100),
                                      (4, 0, 64, 100), (4, 64, 64, 0), (4, 64, 64, 10000001)])
def test_withheld_weight_tile_refusals(M, N, K, us):
    F = 0x100000  # aligned fake device address, never dereferenced on this path
    assert rs.lib().rs_debug_fp8_linear_skip_load(F, K, M, K, N, F, 16384, F, F, 16384, us, None) \
        == rs.RS_ERR_SHAPE
