"""The e4m3 operators where float32 steps, ranges and arguments run out: quotients
halfway between two codes, SiLU of gates far from zero, norms of rows at the ends of the
range; arguments that contradict each other."""
import numpy as np
import pytest
import torch

from gpu_common import F32, dev, log, to_np
from oracle import fp8_ref as F
from test_gpu_fp8 import activations, check_codes, codes_of, given

pytestmark = pytest.mark.gpu
ar = pytest.importorskip("autoround_signsgd_rounding_amd")


# ------------------------------------------------------------------ codes
def want_codes(x, s):
    """Bytes of the e4m3 codes of float32 x over float32 scales s (spread), by division."""
    t = np.asarray(x, F32) / np.asarray(s, F32)
    v = F.e4m3_round(t.astype(np.float64).clip(-448, 448))
    mag = np.searchsorted(F.GRID, np.abs(v)).astype(np.uint8)
    return mag | (np.signbit(t).astype(np.uint8) << 7)


def halfway(rows):
    """Rows of 128 values whose quotients by the row's scale, 1, 3, 5, .., lie halfway between
    two codes (the first value makes the scale; every value is exact in float32)."""
    mid = ((F.GRID[1:] + F.GRID[:-1]) / 2)[:-1]
    s = 2.0 * np.arange(rows) + 1.0
    x = np.concatenate([np.full((rows, 1), 448.0), np.tile(mid, (rows, 1)),
                        np.zeros((rows, 2))], 1) * s[:, None]
    x[:, 2::2] *= -1.0
    assert np.array_equal(x.astype(F32), x)
    return x, s


@pytest.mark.parametrize("rows", [2000, 20000])
@pytest.mark.parametrize("exponent", [-132, -120, -80, 0, 90])
def test_codes_of_quotients_halfway_between_two(rows, exponent):
    """Ties go to the even code, whatever the scale's reciprocal is. The larger call
    takes the kernel of long prompts."""
    log(f"halfway rows={rows} exponent={exponent}")
    x, s = halfway(rows)
    x, s = np.ldexp(x, exponent), np.ldexp(s, exponent)
    keep = s >= 2.0 ** -126
    x, s = x[keep], s[keep]
    X, _ = given(x, "f32")
    q, sc = ar.fp8_quant_act(X)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(to_np(sc)[0], s.astype(F32))
    np.testing.assert_array_equal(codes_of(q), want_codes(x, s[:, None]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(7, 4096), (2200, 1040)])
def test_codes_are_those_of_the_division(M, K, dtype):
    """Every code of both quantizers and of the norm is that of the rounded quotient."""
    log(f"codes by division M={M} K={K} {dtype}")
    rng = np.random.default_rng(M + K)
    X, x = given(activations(rng, M, K), dtype)
    q, s = ar.fp8_quant_act(X)
    wq, ws = ar.fp8_quant_weight(X)
    n = ar.rmsnorm_fp8(X.float(), torch.ones(K, device=dev()), want_y=True)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(codes_of(q), want_codes(x, F.spread_act(to_np(s), K)))
    np.testing.assert_array_equal(codes_of(wq), want_codes(x, F.spread_weight(to_np(ws), M, K)))
    np.testing.assert_array_equal(codes_of(n.q),
                                  want_codes(to_np(n.y), F.spread_act(to_np(n.scale), K)))


# ------------------------------------------------------------------ SiLU
U = 2.0 ** -24


def gated_alone(g, u):
    """Scales and codes [M, KB] of SiLU(g)·u, each alone in a block of zeros."""
    M, KB = g.shape
    x = np.zeros((M, 2, KB, 128), F32)
    x[:, 0], x[:, 1, :, 77] = g[:, :, None], u
    q, s = ar.fp8_quant_act(torch.from_numpy(x.reshape(M, -1)).to(dev()), gate=True)
    torch.cuda.synchronize()
    return to_np(s).T.astype(np.float64), F.e4m3_values(codes_of(q)).reshape(M, KB, 128)[:, :, 77]


def check_gated_alone(g, u):
    """A value alone in its block is 448 times the scale: exp and the reciprocal are good to
    2^-23 each, the sum with 1, exp's correction and two products round once, and so does the
    scale: 9·2^-24, and second orders."""
    g, u = g.astype(F32), u.astype(F32)
    s, code = gated_alone(g, u)
    z = F.silu_mul(np.concatenate([g, u], 1))
    assert np.all(np.abs(z) >= 448 * 2.0 ** -125)         # the scale is a normal number
    err = np.abs(s * 448 / np.abs(z) - 1) / U
    log(f"  worst {err.max():.1f} half units in the last place")
    assert err.max() <= 9.01
    np.testing.assert_array_equal(code, 448.0 * np.sign(z))


@pytest.mark.parametrize("M", [200, 1500])                # 1500: the kernel of long prompts
def test_silu_of_every_gate_to_float32(M):
    log(f"silu of gates M={M}")
    rng = np.random.default_rng(M)
    check_gated_alone(rng.uniform(-82, 60, (M, 16)), rng.uniform(0.5, 2, (M, 16)))
    check_gated_alone(rng.normal(size=(M, 16)), -rng.uniform(0.5, 2, (M, 16)))


@pytest.mark.parametrize("M", [200, 1500])
def test_silu_of_gates_whose_sigmoid_is_no_float32(M):
    """Sigmoids down to 2^-250 times an up half that makes a normal number of them."""
    log(f"silu of far gates M={M}")
    rng = np.random.default_rng(M)
    g = rng.uniform(-170, -80, (M, 16))
    low = np.maximum(g / np.log(2) * -1 - 120, 0)          # z >= 2^-115
    u = 2.0 ** (low + (127 - low) * rng.random((M, 16)))
    check_gated_alone(g, u * rng.choice([-1, 1], (M, 16)))


def test_silu_of_nonfinite_and_huge_gates():
    inf = np.inf
    g = np.array([[inf, inf, -inf, np.nan, 1.0, 1.0, -1000.0, -3e38, 3e38, 1000.0, 0.0]])
    u = np.array([[2.0, -2.0, 2.0, 2.0, inf, np.nan, 3e38, 3e38, 2.0, 2.0, 2.0]])
    s, code = gated_alone(g.astype(F32), u.astype(F32))
    assert np.isposinf(s[0, [0, 1, 4, 8]]).all()
    assert np.all(s[0, [2, 3, 5, 6, 7, 10]] == 1.0)
    assert np.isnan(code[0, [0, 1, 2, 3, 4, 5, 8]]).all() and np.all(code[0, [6, 7, 10]] == 0.0)
    assert s[0, 9] == F32(2000.0) / F32(448.0)


# ------------------------------------------------------------------ RMSNorm
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D", [(40, 16), (7, 512), (3, 2048), (3, 8400), (2, 16400)])
def test_rmsnorm_of_rows_at_the_ends_of_the_range(M, D, dtype):
    """Without an eps a row of subnormal numbers is normalised like any other, and so is one
    near the largest float; a row of zeros is 0/0. Tolerances as for other rows: y is within
    4·2^-24 (and half a step of bf16), codes within 9·2^-24 of x/s."""
    log(f"rmsnorm at the ends M={M} D={D} {dtype}")
    rng = np.random.default_rng(M + D)
    W, w = given(1 + 0.2 * rng.standard_normal(D), dtype)
    for lift in (-146, -131, -127, 120, 125):
        X, x = given(np.ldexp(np.round(4 * rng.standard_normal((M, D))).clip(-7, 7), lift), dtype)
        keep = np.abs(x).max(1) > 0
        o = ar.rmsnorm_fp8(X, W, 0.0, want_y=True)
        torch.cuda.synchronize()
        y = F.rmsnorm(x[keep], w, 0.0)
        half = 2.0 ** -8 if dtype == "bf16" else 0.0
        got = to_np(o.y).astype(np.float64)
        assert np.all(np.abs(got[keep] - y) <= (half + 4 * U) * np.abs(y)), lift
        want = F.act_scales(y)
        q = o.q[torch.from_numpy(keep).to(dev()).nonzero()[:, 0]] if not keep.all() else o.q
        s = o.scale[:, torch.from_numpy(keep).to(dev())]
        check_codes(q, s, y, want, F.spread_act(want, D), np.full(1, 9 * U))
        assert np.isnan(got[~keep]).all()


# ------------------------------------------------------------------ arguments
def products(M=8, N=144, K=256, E=3):
    """The two products as functions of their keywords, on operands of zeros."""
    z = lambda *s, d=torch.float32: torch.zeros(s, dtype=d, device=dev())   # noqa: E731
    f8 = torch.float8_e4m3fn
    x, w, w3 = (z(M, K, d=f8), z(2, M)), (z(N, K, d=f8), z(2, 2)), (z(E, N, K, d=f8), z(E, 2, 2))
    off = z(E + 1, d=torch.int32)
    return (lambda **kw: ar.fp8_gemm(*x, *w, **kw),
            lambda **kw: ar.fp8_gemm_grouped(*x, *w3, off, **kw))


def test_out_dtype_agrees_with_out():
    """An out_dtype beside an out of another type is refused, in both products."""
    types = (torch.float32, torch.bfloat16)
    for call in products():
        for a in types:
            out = torch.empty((8, 144), dtype=a, device=dev())
            assert call(out=out) is out and call(out=out, out_dtype=a) is out
            for b in types + (torch.float16,):
                if b is not a:
                    with pytest.raises(ValueError, match="out_dtype"):
                        call(out=out, out_dtype=b)
                    with pytest.raises(ValueError, match="out_dtype"):
                        call(out=out, out_dtype=b, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
