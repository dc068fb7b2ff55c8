"""Pins of the microscaled-storage oracle: the element tables by the formats'
published values, quantisation by brute force and closed forms, the random
rounding by its mean."""
import itertools

import numpy as np
import pytest
import torch

from oracle import mx


def test_element_tables_are_the_formats():
    assert mx.E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(mx.E4M3, codes.view(torch.float8_e4m3fn).double().numpy())
    codes = torch.arange(124, dtype=torch.uint8)
    assert np.array_equal(mx.E5M2, codes.view(torch.float8_e5m2).double().numpy())
    assert mx.E4M3[-1] == 448 and mx.E5M2[-1] == 57344 and mx.E4M3[1] == 2.0 ** -9


def test_quantise_takes_the_nearest_of_all_codes():
    rng = np.random.default_rng(0)
    W = (rng.standard_normal((6, 64)) * np.exp2(rng.integers(-30, 30, (6, 1)))).astype(np.float32)
    codes, scales = mx.mx4_quantize(W)
    V = mx.mx4_dequant(codes, scales)
    for r, b in itertools.product(range(6), range(2)):
        blk = W[r, 32 * b:32 * b + 32].astype(np.float64)
        s = 2.0 ** (int(scales[r, b]) - 127)
        assert 4 * s <= np.abs(blk).max() < 8 * s
        grid = np.concatenate([-mx.E2M1, mx.E2M1]) * s
        best = np.abs(blk[:, None] - grid).min(1)
        assert np.array_equal(np.abs(blk - V[r, 32 * b:32 * b + 32]), best)
    assert (scales[:, 2:] == 0).all() and scales.shape == (6, 16)


def test_quantise_special_blocks():
    W = np.zeros((1, 160), np.float32)
    W[0, 32:64] = 7.9                 # saturates: e = 0, 7.9 -> 6
    W[0, 64] = 2.0 ** -149            # a subnormal maximum: scale byte 0
    W[0, 100] = np.inf
    W[0, 130:134] = [5.0, 2.5, -1.75, 4.0]  # ties to even: 4, 2, -2
    codes, scales = mx.mx4_quantize(W)
    assert scales[0, :5].tolist() == [0, 127, 0, 255, 127]
    V = mx.mx4_dequant(codes, scales)[0]
    assert (V[:32] == 0).all() and (V[32:64] == 6).all() and (V[64:96] == 0).all() and np.isnan(V[96:128]).all()
    assert V[130:134].tolist() == [4.0, 2.0, -2.0, 4.0]


@pytest.mark.parametrize("table,half,least", [(mx.E4M3, 2.0 ** -4, 2.0 ** -10), (mx.E5M2, 2.0 ** -3, 2.0 ** -17)])
def test_state_round_trips(table, half, least):
    rng = np.random.default_rng(1)
    x = rng.standard_normal(77) * np.exp2(rng.uniform(-12, 0, 77))
    c, s = mx.state_encode_nearest(x, table)
    d = mx.state_decode(c, s, table)
    step = np.repeat(np.exp2(s.astype(float) - 127), 32)[:77]
    assert (np.abs(d - x) <= np.maximum(half * np.abs(x), least * step)).all()
    assert np.array_equal(mx.state_encode_nearest(d, table)[0], c)
    x[3] = np.nan
    assert mx.state_encode_nearest(x, table)[0][3] == 0x7F


@pytest.mark.parametrize("table", [mx.E4M3, mx.E5M2])
@pytest.mark.parametrize("scale", [1.0, -2.0 ** -14])
def test_random_rounding_keeps_the_mean(scale, table):
    x = np.full(32, scale * 0.7137)
    x[0] = 1.0                        # the block's maximum fixes the scale
    got = np.array([mx.state_decode(*mx.state_encode_stochastic(x, mx.random16(32, 3, 11, t), table), table)[1:]
                    for t in range(400)])
    lo, hi = got.min(), got.max()
    assert lo <= x[1] <= hi and len(np.unique(got)) == 2
    # 12400 draws of two values: the mean's standard deviation is at most (hi - lo) / 2 / sqrt(12400); 5 of them
    assert abs(got.mean() - x[1]) < 5 * (hi - lo) / 2 / np.sqrt(got.size)
