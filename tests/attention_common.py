"""Inputs, the oracle's results and bounds of errors of the attention tests."""
import numpy as np
import torch

from gpu_common import dev
from oracle import kv4_ref as R

U = 2.0 ** -24       # half a float32 step, relative


def bf16(x):
    """A bf16 tensor on the GPU and its values in float64."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dev()).to(torch.bfloat16)
    return t, t.double().cpu().numpy()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev())


def keys(rng, n, heads, dim):
    """N(0, 1) with one channel of twenty off zero, as keys have them."""
    k = rng.normal(size=(n, heads, dim))
    big = rng.random((heads, dim)) < 0.05
    return np.where(big, 3 * k + 4 * rng.normal(size=(heads, dim)), k)


def score_error(mag, dim):
    """Bound of a score's error: dim float32 products and sums, the scale times log2 e, and the
    subtraction of the maximum, each half a step of at most mag."""
    return (dim + 6) * U * mag


def out_bound(out, size, mag, dim, n, weight):
    """Bound of |out - exact|: its own rounding to bf16 (2^-8); each weight rounded by `weight`
    and off by a factor of exp(2·score error); n float32 sums and a division."""
    return 2.0 ** -8 * np.abs(out) + size * (
        weight * 1.01 + 2 * np.expm1(2 * score_error(mag, dim)) + (2 * n + 16) * U)[..., None]


def lse_bound(lse, mag, dim, n):
    return 2 * score_error(mag, dim) + (n + 16) * U + 4 * U * np.abs(lse)


def check(got, want, bound, what):
    got = np.asarray(got, np.float64)
    assert np.isfinite(got).all(), what
    worst = np.max(np.abs(got - want) / np.maximum(bound, 1e-300)) if got.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"


def oracle_heads(q, k, v, sees, scale):
    """R.rows over heads: q [n, H, D], k, v [m, Hk, D]; results [n, H, ..]."""
    r = q.shape[1] // k.shape[1]
    per = [R.rows(q[:, h], k[:, h // r], v[:, h // r], sees, scale) for h in range(q.shape[1])]
    return tuple(np.stack(x, 1) for x in zip(*per))
