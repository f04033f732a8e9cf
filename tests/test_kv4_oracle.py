"""Pins of the 4-bit cache's and attention's oracle: hand-computed codes and places, its grid
against the weight quantizer's oracle, its softmax against closed forms."""
import numpy as np
import pytest

import oracle as O
from oracle import kv4_ref as R

F32 = np.float32


def test_grid_by_hand():
    x = np.zeros((1, 32), F32)
    x[0, :4] = [-3.0, 12.0, 0.4, 0.6]              # s = 1, zp = 3
    c, s = R.grid(x, 32)
    assert (s.view(np.uint32) & 15).tolist() == [[3]]
    assert abs(float(s[0, 0]) - 1.0) <= 15 * 2.0 ** -23
    assert c[0, :5].tolist() == [0, 15, 3, 4, 3]
    # all of one sign: zero stays on the grid
    c, s = R.grid(np.linspace(5, 20, 32, dtype=F32)[None], 32)
    assert (s.view(np.uint32) & 15).item() == 0 and c.min() == 4 and c.max() == 15
    # zeros, tiny values
    assert R.grid(np.zeros((1, 32)), 32)[1].item() == 2.0 ** -100
    c, s = R.grid(np.full((1, 32), 1e-40), 32)
    assert s.item() == 2.0 ** -100 and c.max() == 0


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_grid_of_infinities(bad):
    x = np.ones((2, 64), F32)
    x[0, 5] = bad
    c, s = R.grid(x, 32)
    assert np.isnan(s[0, 0]) and np.isfinite(s[0, 1]) and np.isfinite(s[1]).all()
    assert (c[0, :32] == 0).all()
    assert np.isnan(R.grid(np.array([[3e38, -3e38] * 16], F32), 32)[1]).all()


def test_grid_is_the_weight_quantizers():
    """Scales, but for their last bits, and zero-points of asymmetric 4-bit RTN."""
    rng = np.random.default_rng(3)
    x = (rng.normal(size=(64, 128)) * 0.3 + 0.1).astype(F32)
    c, s = R.grid(x, 64)
    codes, scale, zp = O.rtn_quant(x, O.Config(bits=4, group_size=64))[:3]
    assert np.abs(s / scale - 1).max() <= 16 * 2.0 ** -23
    assert ((s.view(np.uint32) & 15) == zp).all()
    assert (c != codes).mean() < 1e-4          # next to a border between two codes


@pytest.mark.parametrize("D,P", [(64, 16), (128, 32)])
def test_places(D, P):
    """Every byte of a page's values has one place; write and held are inverses."""
    at = [R.value_byte(t, b, D // 2) for t in range(P) for b in range(D // 2)]
    assert sorted(at) == list(range(P * D // 2))
    assert R.value_byte(9, 17, 32) == ((1 * 16 + 1) * 8 + 1) * 2 + 1
    rng = np.random.default_rng(D)
    k, v = rng.normal(size=(2, 20, 3, D)).astype(F32)
    codes = np.zeros((3, 2, 3, P, D // 2), np.uint8)
    scale = np.zeros((3, 2, 3, P, D // 32), F32)
    slots = rng.permutation(3 * P)[:20]
    slots[4] = -1
    R.write(codes, scale, k, v, slots)
    for x, got in zip((k, v), R.held(codes, scale, slots)):
        c, s = R.grid(x, 32)
        zp = s.view(np.uint32) & 15
        want = (c.reshape(20, 3, -1, 32).astype(float) - zp[..., None]) * s.astype(float)[..., None]
        want[4] = 0
        np.testing.assert_array_equal(got, want.reshape(20, 3, D))


def test_softmax_by_hand():
    q, k, v = np.array([[2.0, 0.0]]), np.array([[0.0, 1.0], [np.log(3.0), 0.0]]), np.array([[1.0], [5.0]])
    o, lse, size, mag = R.rows(q, k, v, np.ones((1, 2), bool), 0.5)
    np.testing.assert_allclose(o, [[(1 + 3 * 5) / 4]])
    np.testing.assert_allclose(lse, [np.log(4.0)])
    np.testing.assert_allclose([size[0, 0], mag[0]], [4.0, np.log(3.0)])
    o, lse, _, _ = R.rows(q, k, v, np.zeros((1, 2), bool), 0.5)
    assert o[0, 0] == 0 and lse[0] == -np.inf
    assert R.causal(2, 4).tolist() == [[True, True, True, False], [True] * 4]
    assert R.causal(3, 1).tolist() == [[False], [False], [True]]
