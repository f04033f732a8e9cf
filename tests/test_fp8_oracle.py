"""Pins of the e4m3 oracle: its value table and rounding against torch's
float8_e4m3fn, its scales and products against hand-computed values."""
import numpy as np
import torch

from oracle import fp8_ref as F


def test_values_of_every_code():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(F.e4m3_values(codes).astype(np.float32), want)
    assert F.GRID[-1] == 448.0 and len(F.GRID) == 127


def test_rounding():
    rng = np.random.default_rng(0)
    mid = (F.GRID[1:] + F.GRID[:-1]) / 2                     # every tie
    t = np.concatenate([F.GRID, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9),
                        rng.uniform(0, 448, 2000), 2.0 ** rng.uniform(-12, 8.8, 2000)])
    t = np.concatenate([t, -t]).astype(np.float32)
    want = torch.from_numpy(t).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(F.e4m3_round(t).astype(np.float32), want)


def test_scales_by_hand():
    x = np.zeros((2, 144))
    x[0, 3], x[0, 130], x[1, 7] = -896.0, 4.48, 1e-44
    s = F.act_scales(x)
    assert s.shape == (2, 2)
    np.testing.assert_allclose(s, [[2.0, 2.0 ** -126], [0.01, 1.0]])
    w = np.zeros((1, 129, 16))
    w[0, 128, 15] = 44.8
    np.testing.assert_allclose(F.weight_scales(w), [[[1.0], [0.1]]])
    assert F.spread_act(s, 144)[0, 127] == 2.0 and F.spread_act(s, 144)[0, 128] == 0.01
    assert F.spread_weight(F.weight_scales(w), 129, 16)[0, 128, 0] == 44.8 / 448


def test_products_by_hand():
    xq, wq = np.ones((1, 144)), np.full((130, 144), 2.0)
    xs, ws = np.array([[1.0], [10.0]]), np.array([[1.0, 1.0], [0.5, 3.0]])
    y, s = F.product(xq, xs, wq, ws)
    assert y[0, 0] == 128 * 2 + 16 * 2 * 10 and y[0, 129] == 128 + 16 * 2 * 10 * 3
    np.testing.assert_array_equal(y, s)
    out = np.full((4, 130), 7.0)
    g, _ = F.grouped_product(xq, xs, wq[None], ws[None], [1, 3], [0, 0, -1, 0], out)
    np.testing.assert_array_equal(g[[0, 3]], 7.0)
    np.testing.assert_array_equal(g[1], y[0])
    np.testing.assert_array_equal(g[2], 0.0)


def test_norm_and_gate_by_hand():
    y = F.rmsnorm([[3.0, 4.0]], [1.0, 2.0], 0.0)
    np.testing.assert_allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])
    np.testing.assert_allclose(F.silu_mul([[0.0, np.log(3.0), 5.0, 2.0]]),
                               [[0.0, 1.5 * np.log(3.0)]])
