"""The 64-bit definitions the GPU tests compare with, pinned by hand values and by an
exhaustive search over the e4m3 values (CPU)."""
import math

import pytest
import torch

import fp8_ref as R


def all_e4m3():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    return v[torch.isfinite(v)]


def test_e4m3_is_the_nearest_value_with_ties_to_even():
    vals, idx = torch.sort(torch.unique(all_e4m3()))
    g = torch.Generator().manual_seed(0)
    x = torch.cat([(torch.rand(4000, generator=g, dtype=R.F64) * 2 - 1) * 448.0,
                   torch.randn(4000, generator=g, dtype=R.F64) * 0.01, vals,
                   (vals[1:] + vals[:-1]) / 2])
    got = R.e4m3(x)
    d = (x[:, None] - vals[None]).abs()
    best = d.min(1).values
    assert torch.equal((x - got).abs(), best)
    assert torch.isin(got, vals).all()
    tie = (d == best[:, None]).sum(1) == 2
    assert tie.any()
    mant = (got[tie] / R.e4m3_step(got[tie])).abs()
    assert (mant % 2 == 0).all()


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0001, 1), (224.0, -1), (1.0, -8),
                                    (1.75, -8), (1.7500001, -7), (0.0, -127), (2.0 ** -140, -127),
                                    (3.4e38, 120), (1.75 * 2.0 ** 127, 119)])
def test_block_exponent(amax, e):
    x = torch.zeros(1, 128, dtype=R.F64)
    x[0, 17] = -amax
    assert R.block_exponents(x).item() == e


def test_blocks_do_not_mix_and_the_last_may_be_short():
    x = torch.ones(1, 130, dtype=R.F64)
    x[0, 128] = 1000.0
    assert R.block_exponents(x).tolist() == [[-8, 2]]
    assert R.quantized(x)[0, 128:].tolist() == [1024.0, 1.0]  # step 64 at 1000 / 4 = 250 -> 16 * 4
    assert R.quantized(torch.tensor([[math.inf, 3.0, math.nan]], dtype=R.F64))[0, 1] == 3.0


def test_scale_places_are_distinct_and_inside():
    at = R.scale_index(300, 1200)
    assert at.unique().numel() == at.numel() and int(at.max()) < 3 * 3 * 512


def test_layer_norm_gradient_against_differences():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 7, generator=g, dtype=R.F64)
    gam, bet = torch.randn(7, generator=g, dtype=R.F64), torch.randn(7, generator=g, dtype=R.F64)
    dy = torch.randn(3, 7, generator=g, dtype=R.F64)
    dx, dg, db = R.layer_norm_grad(dy, x, gam, 1e-6)
    f = lambda x_, g_, b_: (R.layer_norm(x_, g_, b_, 1e-6)[0] * dy).sum()  # noqa: E731
    h = 1e-6
    for i in range(3):
        for j in range(7):
            d = torch.zeros_like(x)
            d[i, j] = h
            assert abs((f(x + d, gam, bet) - f(x - d, gam, bet)) / (2 * h) - dx[i, j]) < 1e-7
    for j in range(7):
        d = torch.zeros_like(gam)
        d[j] = h
        assert abs((f(x, gam + d, bet) - f(x, gam - d, bet)) / (2 * h) - dg[j]) < 1e-7
        assert abs((f(x, gam, bet + d) - f(x, gam, bet - d)) / (2 * h) - db[j]) < 1e-7
