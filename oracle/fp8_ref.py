"""The e4m3 operators in float64: quantizers, RMSNorm with an e4m3 output and the
block-scaled products, from their definitions in include/autoround_hip.h."""
import numpy as np

BLOCK = 128


def _grid():
    """The non-negative e4m3 values in order: subnormals m·2^-9, then (1 + m/8)·2^(e-7) up to 448."""
    return np.array([m * 2.0 ** -9 for m in range(8)] +
                    [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])


GRID = _grid()                      # GRID[code & 0x7F] is a code's magnitude


def e4m3_values(codes):
    """uint8 codes -> float64 values (0x7F and 0xFF are NaN)."""
    codes = np.asarray(codes, np.uint8)
    v = np.append(GRID, np.nan)[codes & 0x7F]
    return np.where(codes & 0x80, -v, v)


def e4m3_round(t):
    """Nearest e4m3 value of finite |t| <= 464, ties to the even code."""
    t = np.asarray(t, np.float64)
    a = np.abs(t)
    hi = np.searchsorted(GRID, a).clip(1, len(GRID) - 1)
    lo = hi - 1
    dl, dh = a - GRID[lo], GRID[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.copysign(np.where(up, GRID[hi], GRID[lo]), t)


def blocks(n):
    return -(-n // BLOCK)


def scale_of(amax):
    amax = np.asarray(amax, np.float64)
    return np.where(amax == 0, 1.0, np.maximum(amax / 448.0, 2.0 ** -126))


def act_scales(x):
    """[KB, M] scales of x [M, K]."""
    M, K = x.shape
    a = np.abs(np.asarray(x, np.float64))
    return np.stack([scale_of(a[:, j * BLOCK:(j + 1) * BLOCK].max(1)) for j in range(blocks(K))])


def weight_scales(w):
    """[E, NB, KB] scales of w [E, N, K]."""
    a = np.abs(np.asarray(w, np.float64))
    E, N, K = a.shape
    s = np.empty((E, blocks(N), blocks(K)))
    for i in range(blocks(N)):
        for j in range(blocks(K)):
            s[:, i, j] = scale_of(a[:, i * BLOCK:(i + 1) * BLOCK,
                                    j * BLOCK:(j + 1) * BLOCK].max((1, 2)))
    return s


def spread_act(s, K):
    """[KB, M] -> [M, K]."""
    return np.repeat(s.T, BLOCK, axis=1)[:, :K]


def spread_weight(s, N, K):
    """[..., NB, KB] -> [..., N, K]."""
    return np.repeat(np.repeat(s, BLOCK, axis=-2)[..., :N, :], BLOCK, axis=-1)[..., :K]


def silu_mul(x):
    """SiLU of the first half of the channels times the second half."""
    g, u = np.split(np.asarray(x, np.float64), 2, axis=1)
    return g / (1.0 + np.exp(-g)) * u


def rmsnorm(v, w, eps):
    v = np.asarray(v, np.float64)
    return v / np.sqrt((v * v).mean(1, keepdims=True) + eps) * np.asarray(w, np.float64)


def product(xq, xs, wq, ws):
    """(Y, S): the product in float64 and the sum of its terms' magnitudes.
    xq [M, K], wq [N, K] e4m3 values, xs [KB, M], ws [NB, KB]."""
    N, K = wq.shape
    x = xq * spread_act(np.asarray(xs, np.float64), K)
    w = wq * spread_weight(np.asarray(ws, np.float64), N, K)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def product_bound(K):
    """Largest error of a float32 result over the sum of the terms' magnitudes.
    A term's product is exact; a block adds 128 terms to zero, its sum and the
    scale product (rounded once) meet the accumulator in one rounding, and up to
    KB + 8 accumulations follow, each rounding by at most 2^-23 of what it holds
    (twice the half step of float32: the matrix unit need not round to nearest).
    Where a bf16 result lets the e4m3 unit add a block in its own narrower sum, that
    sum is off by up to 4e-5 of its size for products of like sizes; the magnitudes of
    128 terms add up to several times the size of a sum of random signs, so the bound
    holds there too. Products of very different sizes: unit_bound()."""
    return (BLOCK + blocks(K) + 10) * 2.0 ** -23


def unit_bound(xq, xs, wq, ws):
    """What the e4m3 unit may lose beyond product_bound() in a bf16 result. It adds
    the products of 8 neighbouring channels first, cut off 13 bits below the largest
    one's exponent: up to 7 of them lose less than 2^-13 of that one each."""
    M, (N, K) = xq.shape[0], wq.shape
    x = np.abs(xq * spread_act(np.asarray(xs, np.float64), K))
    w = np.abs(wq * spread_weight(np.asarray(ws, np.float64), N, K))
    lost = np.zeros((M, N))
    for k in range(0, K, 8):
        lost += (x[:, None, k:k + 8] * w[None, :, k:k + 8]).max(2)
    return lost * 7 * 2.0 ** -13


def grouped_product(xq, xs, wq, ws, offsets, row_index, out):
    """Rows of `out` replaced by their expert's product; (Y, S) as product()."""
    y, s = np.array(out, np.float64), np.zeros(np.shape(out))
    R = y.shape[0]
    rows = np.arange(R) if row_index is None else np.asarray(row_index)
    for e in range(wq.shape[0]):
        r = np.arange(offsets[e], offsets[e + 1])
        if len(r) == 0:
            continue
        src = rows[r]
        ok = (src >= 0) & (src < xq.shape[0])
        y[r] = 0.0
        y[r[ok]], s[r[ok]] = product(xq[src[ok]], xs[:, src[ok]], wq[e], ws[e])
    return y, s
