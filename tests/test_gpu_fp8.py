"""GPU parity of the e4m3 operators (quantizers, RMSNorm with an e4m3 output,
block-scaled products dense and by expert) against the float64 oracle.

Tolerances. A code may differ from the nearest e4m3 value of the exact x/s by
what float32 moved x/s: |code - x/s| <= (distance to the nearest value) +
2·rel·|x/s|, rel being the relative error of x and of s together (the factor
for a tie crossed on the way). s = amax/448 and 1/s and x·(1/s) round once each
(3·2^-24); the norm's y = (v·r)·w adds 3·2^-24 and as much again through amax;
SiLU(g)·u adds (2|g| + 9)·2^-24: the exponent's argument and the constant in it
move exp by 2|g|·2^-24, exp and the reciprocal are good to 2^-23 each, the sum
and the two products round once. The products' bound is fp8_ref.product_bound
over the sum of the terms' magnitudes, and half a step of bf16 (2^-8) where the
output is rounded to it."""
import numpy as np
import pytest
import torch

import synth
from gpu_common import F32, bf16_dev, bf16_bits_of, dev, log, to_np
from oracle import fp8_ref as F

pytestmark = pytest.mark.gpu
ar = pytest.importorskip("autoround_signsgd_rounding_amd")

U = 2.0 ** -24
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


def given(x, dtype):
    """(device tensor, the float64 values it holds)."""
    x = np.asarray(x, F32)
    if dtype == "bf16":
        bits = synth.f32_to_bf16_bits(x)
        return bf16_dev(bits), synth.bf16_bits_to_f32(bits).astype(np.float64)
    return torch.from_numpy(np.ascontiguousarray(x)).to(dev()), x.astype(np.float64)


def codes_of(q):
    return q.view(torch.uint8).cpu().numpy()


def activations(rng, M, K):
    x = rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.02, 20.0, 1.0)
    if M > 2:
        x[1] = 0.0                         # a row of zero blocks
        x[2, : K // 2] *= 1e-6
    return x


def check_codes(q, s, exact, want_s, s_spread, rel):
    """Scales within rel, codes next to exact/scale within what rel allows."""
    got_s = to_np(s).astype(np.float64)
    assert got_s.shape == want_s.shape
    err = np.abs(got_s - want_s)
    assert np.all(err <= rel.max() * want_s), (err / want_s).max()
    t = exact / s_spread
    v = F.e4m3_values(codes_of(q))
    slack = np.abs(F.e4m3_round(t) - t) + 2 * rel * np.abs(t) + 1e-30
    bad = np.abs(v - t) > slack
    assert not bad.any(), (bad.sum(), v[bad][:4], t[bad][:4])


ACT = [(1, 16), (1, 4096), (3, 144), (33, 128), (300, 1040), (2, 11008), (70, 272), (2200, 512)]


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", ACT)
def test_quant_act(M, K, dtype, gate):
    log(f"quant_act M={M} K={K} {dtype} gate={gate}")
    rng = np.random.default_rng(M * 7 + K)
    X, x = given(activations(rng, M, 2 * K if gate else K), dtype)
    q, s = ar.fp8_quant_act(X, gate=gate)
    torch.cuda.synchronize()
    assert q.dtype == F8 and tuple(q.shape) == (M, K) and tuple(s.shape) == (F.blocks(K), M)
    exact = F.silu_mul(x) if gate else x
    want = F.act_scales(exact)
    rel = (2 * np.abs(x[:, :K]).max() + 9 if gate else 0) * U + 3 * U
    check_codes(q, s, exact, want, F.spread_act(want, K), np.full(1, 2 * rel))


@pytest.mark.parametrize("M", [3, 2200])
def test_quant_act_of_gates_far_below_zero(M):
    """Sigmoids below 2^-126 (a gate under -87.3) times a large up half: the
    result is a normal number, in blocks of nothing else. The exponential's argument
    is off by |gate| U, the sigmoid as a subnormal of 2^-128 by 2^-22."""
    log(f"quant_act of gates far below zero M={M}")
    rng = np.random.default_rng(M)
    x = np.concatenate([rng.uniform(-88.7, -86.0, (M, 256)),
                        1e30 * rng.uniform(0.5, 1.0, (M, 256))], 1)
    X, x = given(x, "f32")
    q, s = ar.fp8_quant_act(X, gate=True)
    torch.cuda.synchronize()
    exact = F.silu_mul(x)
    want = F.act_scales(exact)
    check_codes(q, s, exact, want, F.spread_act(want, 256), np.full(1, 2 * (2 * 88.7 + 16) * U))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,N,K", [(1, 1, 16), (3, 130, 272), (1, 256, 512), (9, 128, 128),
                                   (2, 77, 1040)])
def test_quant_weight(E, N, K, dtype):
    log(f"quant_weight E={E} N={N} K={K} {dtype}")
    rng = np.random.default_rng(E + N + K)
    w = 0.02 * rng.standard_normal((E, N, K))
    w[E - 1, :128, :128] = 0.0             # a zero block
    W, x = given(w, dtype)
    q, s = ar.fp8_quant_weight(W)
    q2, s2 = ar.fp8_quant_weight(W[0])
    torch.cuda.synchronize()
    want = F.weight_scales(x)
    check_codes(q, s, x, want, F.spread_weight(want, N, K), np.full(1, 3 * U))
    assert torch.equal(q2.view(torch.uint8), q[0].view(torch.uint8)) and torch.equal(s2, s[0])


def test_quant_of_extreme_values():
    """Blocks of tiny values keep a normal scale; a NaN stays in its place; an
    infinity makes its block's scale infinite, its own code NaN, the others 0."""
    x = np.ones((4, 256), F32)
    x[0, :128] = 1e-40
    x[1, 5] = np.nan
    x[2, 200] = -np.inf
    x[3, 0] = 3.3e38
    q, s = ar.fp8_quant_act(torch.from_numpy(x).to(dev()))
    torch.cuda.synchronize()
    v, s = F.e4m3_values(codes_of(q)), to_np(s)
    assert s[0, 0] == 2.0 ** -126 and np.isposinf(s[1, 2])
    assert s[0, 1] == s[1, 0] == F32(1) / F32(448)
    assert np.isnan(v[1, 5]) and np.isnan(v).sum() == 2
    assert np.isnan(v[2, 200]) and np.all(np.delete(v[2, 128:], 72) == 0)
    assert v[3, 0] == 448.0 and np.all(v[3, 1:128] == 0) and np.all(v[1, :5] == 448.0)


NORM = [(1, 16), (1, 4096), (3, 144), (5, 1024), (70, 1040), (9, 4112), (4, 8192), (3, 8208),
        (2, 20000), (1100, 256), (37, 128), (6, 2048)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D", NORM)
def test_rmsnorm(M, D, dtype):
    log(f"rmsnorm M={M} D={D} {dtype}")
    rng = np.random.default_rng(M + D)
    X, x = given(activations(rng, M, D), dtype)
    Rs, r = given(activations(rng, M, D), dtype)
    W, w = given(1 + 0.2 * rng.standard_normal(D), dtype)
    for residual in (None, Rs):
        o = ar.rmsnorm_fp8(X, W, 1e-5, residual=residual, want_y=True)
        torch.cuda.synchronize()
        v = x
        if residual is None:
            assert o.h is None
        else:
            v32 = x.astype(F32) + r.astype(F32)
            if dtype == "bf16":
                bits = synth.f32_to_bf16_bits(v32)
                np.testing.assert_array_equal(bf16_bits_of(o.h), bits)
                v = synth.bf16_bits_to_f32(bits).astype(np.float64)
            else:
                np.testing.assert_array_equal(to_np(o.h), v32)
                v = v32.astype(np.float64)
        y = F.rmsnorm(v, w, float(F32(1e-5)))
        half = 2.0 ** -8 if dtype == "bf16" else 0.0
        assert np.all(np.abs(to_np(o.y) - y) <= (half + 4 * U) * np.abs(y))
        want = F.act_scales(y)
        check_codes(o.q, o.scale, y, want, F.spread_act(want, D), np.full(1, 9 * U))


def test_rmsnorm_of_large_values_and_in_place():
    """Squares past float32's range; the residual stream updated in place gives
    the same bits as into a new tensor, at widths held in registers and one that
    is read twice."""
    for D in (512, 8400, 16400):
        rng = np.random.default_rng(D)
        X, _ = given(1e30 * rng.standard_normal((5, D)), "f32")
        Rs, _ = given(1e30 * rng.standard_normal((5, D)), "f32")
        W, _ = given(np.ones(D), "f32")
        o = ar.rmsnorm_fp8(X, W, residual=Rs, want_y=True)
        for x_, r_, kept in ((X, Rs.clone(), "r"), (X.clone(), Rs, "x")):
            kept = r_ if kept == "r" else x_
            a = ar.rmsnorm_fp8(x_, W, residual=r_, h_out=kept)
            torch.cuda.synchronize()
            assert a.h is kept and torch.equal(kept, o.h) and torch.equal(a.scale, o.scale)
            assert torch.equal(a.q.view(torch.uint8), o.q.view(torch.uint8))
        y = to_np(o.y).astype(np.float64)
        assert np.all(np.isfinite(y)) and np.allclose((y * y).mean(1), 1.0, atol=1e-5)


# ------------------------------------------------------------------ products
def random_codes(rng, shape):
    """Codes of every magnitude but NaN, most of them large."""
    c = (448 * rng.standard_normal(shape) / 4).clip(-448, 448).astype(F32)
    return torch.from_numpy(c).to(dev()).to(F8)


def operands(rng, T, E, N, K):
    xq, wq = random_codes(rng, (T, K)), random_codes(rng, (E, N, K))
    xs = torch.from_numpy(rng.uniform(0.5, 2.0, (F.blocks(K), T)).astype(F32) * 0.01).to(dev())
    ws = torch.from_numpy(rng.uniform(0.5, 2.0, (E, F.blocks(N), F.blocks(K))).astype(F32)
                          * 1e-3).to(dev())
    return xq, xs, wq, ws


def values(xq, xs, wq, ws):
    return (F.e4m3_values(codes_of(xq)), to_np(xs).astype(np.float64),
            F.e4m3_values(codes_of(wq)), to_np(ws).astype(np.float64))


def check_product(got, y, s, K, out):
    tol = F.product_bound(K) * s
    if out == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(y)
    err = np.abs(got.astype(np.float64) - y)
    assert np.all(err <= tol), (err.max(), np.argwhere(err > tol)[:4])


OUT = {"bf16": BF16, "f32": torch.float32}
GEMM = [
    # M, N, K, out
    (1, 1, 16, "f32"), (1, 4096, 4096, "bf16"), (1, 100, 128, "f32"), (2, 130, 144, "bf16"),
    (7, 513, 1040, "f32"), (16, 256, 2048, "bf16"), (17, 300, 400, "f32"), (33, 4, 128, "bf16"),
    (64, 1000, 720, "f32"), (65, 129, 272, "bf16"), (100, 22, 1984, "bf16"),
    (128, 256, 256, "f32"), (130, 514, 384, "bf16"), (256, 512, 1024, "f32"),
    (300, 2050, 1360, "f32"), (513, 260, 112, "bf16"), (1000, 1030, 528, "bf16"),
    (2048, 768, 640, "bf16"), (3000, 64, 256, "f32"),
    # more than 64 and 128 blocks of K, whole and short last blocks, on every path
    (5, 40, 17008, "bf16"), (40, 130, 17008, "bf16"), (300, 200, 11008, "f32"),
    (600, 1100, 8336, "bf16"), (4100, 4200, 8464, "bf16"),
    # large tiles with rows of Y that start at any 2 bytes, and at any 4
    (6200, 4831, 528, "bf16"), (6200, 4830, 272, "bf16"),
]


@pytest.mark.parametrize("M,N,K,out", GEMM)
def test_gemm(M, N, K, out):
    log(f"fp8_gemm M={M} N={N} K={K} {out}")
    rng = np.random.default_rng(M + N + K)
    xq, xs, wq, ws = operands(rng, M, 1, N, K)
    Y = ar.fp8_gemm(xq, xs, wq[0], ws[0], out_dtype=OUT[out])
    again = ar.fp8_gemm(xq, xs, wq[0], ws[0], out_dtype=OUT[out])
    torch.cuda.synchronize()
    assert torch.equal(Y, again)
    x, s, w, t = values(xq, xs, wq, ws)
    y, mag = F.product(x, s, w[0], t[0])
    check_product(to_np(Y), y, mag, K, out)


@pytest.mark.parametrize("M,N,K", [(4096, 4096, 4096), (16, 29568, 8192), (333, 11008, 4096)])
def test_gemm_full_size_sampled(M, N, K):
    """Real layer sizes, compared on sampled rows and columns."""
    log(f"fp8_gemm M={M} N={N} K={K} sampled")
    g = torch.Generator(device=dev())
    g.manual_seed(M + N)
    xq, xs = ar.fp8_quant_act(torch.randn((M, K), generator=g, device=dev()))
    wq, ws = ar.fp8_quant_weight(0.02 * torch.randn((N, K), generator=g, device=dev()))
    Y = ar.fp8_gemm(xq, xs, wq, ws, out_dtype=torch.float32)
    torch.cuda.synchronize()
    r = torch.randperm(M, generator=g, device=dev())[:64].sort().values
    c = torch.cat([torch.arange(N - 128, N, device=dev()),      # two whole blocks
                   torch.arange(128 * 5, 128 * 6, device=dev())])
    x, s, w, t = values(xq.view(torch.uint8)[r], xs[:, r], wq.view(torch.uint8)[c],
                        ws[[N // 128 - 1, 5]])
    y, mag = F.product(x, s, w, t)
    check_product(to_np(Y[r][:, c]), y, mag, K, "f32")


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", [(3, 100), (200, 140), (700, 300)])
def test_gemm_of_outliers_that_cancel(M, N, out):
    """Two products of 448^2 in each block of K cancel, among products near 1: a bf16
    result may lose what the matrix unit cuts off, a float32 one nothing of it."""
    log(f"fp8_gemm outliers that cancel M={M} N={N} {out}")
    rng = np.random.default_rng(M)
    K = 400
    xq, xs, wq, ws = operands(rng, M, 1, N, K)
    x, w = rng.standard_normal((M, K)), rng.standard_normal((N, K))
    for j in range(F.blocks(K)):
        p, q = 128 * j + rng.choice(min(128, K - 128 * j), 2, replace=False)
        x[:, p], x[:, q], w[:, p], w[:, q] = 448.0, -448.0, 448.0, 448.0
    xq.copy_(torch.from_numpy(x).to(dev()).to(F8))
    wq.copy_(torch.from_numpy(w).to(dev()).to(F8)[None])
    Y = to_np(ar.fp8_gemm(xq, xs, wq[0], ws[0], out_dtype=OUT[out])).astype(np.float64)
    a, s, b, t = values(xq, xs, wq, ws)
    y, mag = F.product(a, s, b[0], t[0])
    tol = F.product_bound(K) * mag
    if out == "bf16":
        tol = tol + F.unit_bound(a, s, b[0], t[0]) + 2.0 ** -8 * np.abs(y)
    assert np.all(np.abs(Y - y) <= tol), (np.abs(Y - y) / tol).max()


def test_gemm_zero_and_nonfinite():
    """A NaN code reaches its row (or column) only; an infinite scale too."""
    rng = np.random.default_rng(1)
    for M in (3, 200):
        N, K = 140, 256
        xq, xs, wq, ws = operands(rng, M, 1, N, K)
        clean = ar.fp8_gemm(xq, xs, wq[0], ws[0], out_dtype=torch.float32)
        xq.view(torch.uint8)[1, 9] = 0x7F
        wq.view(torch.uint8)[0, 130, 200] = 0xFF
        xs[1, 2] = float("inf")
        Y = to_np(ar.fp8_gemm(xq, xs, wq[0], ws[0], out_dtype=torch.float32))
        bad = np.zeros((M, N), bool)
        bad[1] = bad[2] = True
        bad[:, 130] = True
        assert not np.isfinite(Y[bad]).any()
        np.testing.assert_array_equal(Y[~bad], to_np(clean)[~bad])


# counts per expert, N, K, gather, out
GROUPED = [
    ([3, 0, 1, 5], 64, 128, False, "f32"),
    ([0, 0, 7, 0], 130, 144, True, "bf16"),
    ([1] * 70 + [0, 2], 100, 272, True, "f32"),
    ([16, 17, 15, 33], 513, 400, False, "bf16"),
    ([100, 0, 300, 1], 260, 528, True, "f32"),
    ([700], 129, 256, True, "bf16"),
    ([513, 2, 0, 255, 257], 384, 640, False, "f32"),
    ([2000, 0, 3, 1100], 300, 384, True, "bf16"),
    ([0, 0, 0], 64, 128, False, "f32"),
    # more experts than a wave has lanes, and than four times that
    ([1, 0, 2] * 100, 130, 144, True, "bf16"),
    ([70, 0, 3] * 90, 140, 272, False, "bf16"),
    ([0] * 299 + [40], 64, 128, True, "f32"),
]


def grouped_case(counts, N, K, gather, seed, before=0, after=0):
    """Operands, offsets and index; `before` and `after` rows belong to no expert."""
    rng = np.random.default_rng(seed)
    E = len(counts)
    off = before + np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(off[-1]) + after
    T = max(R // 2, 1) + 3 if gather else R
    ops = operands(rng, T, E, N, K)
    idx = None
    if gather:
        idx = rng.integers(0, T, R).astype(np.int32)        # repeats among them
        idx[: R // 7] = idx[0] if R else 0
    to = lambda a: None if a is None else torch.from_numpy(a).to(dev())   # noqa: E731
    return ops, off, idx, to(off), to(idx), R


@pytest.mark.parametrize("counts,N,K,gather,out", GROUPED)
def test_grouped(counts, N, K, gather, out):
    log(f"fp8_gemm_grouped counts={counts[:5]}.. N={N} K={K} gather={gather} {out}")
    ops, off, idx, offd, idxd, R = grouped_case(counts, N, K, gather, N + K, before=2, after=37)
    if gather and R > 6:
        idx[3], idx[5] = -1, ops[0].shape[0]                 # rows that name no token
        idxd = torch.from_numpy(idx).to(dev())
    Y = torch.full((R, N), 5.0, dtype=OUT[out], device=dev())
    ar.fp8_gemm_grouped(*ops, offd, row_index=idxd, out=Y)
    torch.cuda.synchronize()
    y, mag = F.grouped_product(*values(*ops), off, idx, np.full((R, N), 5.0))
    got = to_np(Y)
    check_product(got, y, mag, K, out)
    np.testing.assert_array_equal(got[: off[0]], 5.0)
    np.testing.assert_array_equal(got[off[-1]:], 5.0)


@pytest.mark.parametrize("off", [[-5, 4, 9, 10 ** 9], [0, 30, 10, 60], [60, 0, 60, 0]])
def test_grouped_bad_offsets_stay_inside(off):
    """Offsets outside [0, R] or decreasing: rows are unspecified, but nothing
    around Y changes and the call ends."""
    R, N, K, G = 60, 130, 256, 16
    rng = np.random.default_rng(2)
    ops = operands(rng, R, 3, N, K)
    big = torch.full((R + 2 * G, N), 3.0, device=dev())
    Y = big[G:G + R]
    ar.fp8_gemm_grouped(*ops, torch.tensor(off, dtype=torch.int32, device=dev()), out=Y)
    torch.cuda.synchronize()
    assert torch.all(big[:G] == 3.0) and torch.all(big[G + R:] == 3.0)


@pytest.mark.parametrize("counts,N,K,out", [
    ([20, 0, 13], 140, 272, "f32"), ([1, 1], 40, 256, "bf16"), ([700, 40], 260, 256, "bf16"),
    ([400], 300, 528, "f32"), ([6000], 4100, 128, "bf16")])
def test_grouped_rows_without_a_token_beside_nonfinite_weights(counts, N, K, out):
    """A row whose index names no token is zero, also where its expert's weight holds
    NaN codes and infinite scales; the other rows show them."""
    log(f"fp8_gemm_grouped no token, nonfinite W {counts} N={N} K={K} {out}")
    ops, off, idx, offd, _, R = grouped_case(counts, N, K, True, 77)
    idx[::3] = -1
    idx[1::7] = ops[0].shape[0]
    ops[2].view(torch.uint8)[:, N // 2, K - 3] = 0x7F
    ops[3][:, 0, 0] = float("inf")
    Y = to_np(ar.fp8_gemm_grouped(*ops, offd, row_index=torch.from_numpy(idx).to(dev()),
                                  out_dtype=OUT[out]))
    none = (idx < 0) | (idx >= ops[0].shape[0])
    assert np.all(Y[none] == 0.0)
    assert np.isnan(Y[~none][:, N // 2]).all() and not np.isfinite(Y[~none][:, 0]).any()


def test_empty_calls():
    z = lambda *s, d=torch.float32: torch.zeros(s, dtype=d, device=dev())   # noqa: E731
    q, s = ar.fp8_quant_act(z(0, 64))
    assert tuple(q.shape) == (0, 64) and tuple(s.shape) == (1, 0)
    assert ar.rmsnorm_fp8(z(0, 32), z(32)).q.shape == (0, 32)
    wq, ws = ar.fp8_quant_weight(z(2, 48, 64))
    assert ar.fp8_gemm(q, s, wq[0], ws[0]).shape == (0, 48)
    off = torch.zeros(3, dtype=torch.int32, device=dev())
    assert ar.fp8_gemm_grouped(q, s, wq, ws, off).shape == (0, 48)
    idx = torch.zeros(0, dtype=torch.int32, device=dev())
    q1, s1 = ar.fp8_quant_act(z(4, 64))
    assert ar.fp8_gemm_grouped(q1, s1, wq, ws, off, row_index=idx).shape == (0, 48)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ graphs, streams, chains
def test_grouped_under_graph_capture():
    """A captured call replayed with other offsets and indices in the same
    buffers, eager work in between, equals the eager call on them every time."""
    for counts, more in (([2, 0, 5, 1], [0, 4, 0, 4]), ([200, 90, 0, 300], [10, 300, 280, 0])):
        ops, _, _, offd, idxd, R = grouped_case(counts, 320, 384, True, 11)
        Y = torch.zeros((R, 320), device=dev())
        ar.fp8_gemm_grouped(*ops, offd, row_index=idxd, out=Y)
        torch.cuda.synchronize()
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                ar.fp8_gemm_grouped(*ops, offd, row_index=idxd, out=Y)
        torch.cuda.synchronize()
        for i in range(4):
            c = counts if i % 2 else more
            offd.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(c)]).astype(np.int32)))
            idxd.add_(1).remainder_(ops[0].shape[0])
            Y.fill_(float(i))
            want = torch.full_like(Y, float(i))
            ar.fp8_gemm_grouped(*ops, offd, row_index=idxd, out=want)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(Y, want), i


@pytest.mark.parametrize("M", [1, 300])
def test_chain_under_graph_capture(M):
    """norm -> gate|up -> SiLU·mul codes -> down, captured as a decode step is."""
    D, FF = 256, 384
    rng = np.random.default_rng(M)
    X, _ = given(activations(rng, M, D), "bf16")
    Rs, _ = given(activations(rng, M, D), "bf16")
    W, _ = given(np.ones(D), "bf16")
    wgu, wd = (ar.fp8_quant_weight(given(0.05 * rng.standard_normal(s), "bf16")[0])
               for s in ((2 * FF, D), (D, FF)))

    def step():
        n = ar.rmsnorm_fp8(X, W, residual=Rs)
        z = ar.fp8_quant_act(ar.fp8_gemm(n.q, n.scale, *wgu), gate=True)
        return n.h, ar.fp8_gemm(*z, *wd)

    eager = step()
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            kept = step()
    torch.cuda.synchronize()
    for _ in range(4):
        for t in kept:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(kept, eager):
            assert torch.equal(a, b)
        step()
        torch.cuda.synchronize()


def test_calls_on_another_stream():
    """`stream=` runs and allocates there; two streams at once keep apart."""
    rng = np.random.default_rng(4)
    a, b = operands(rng, 70, 1, 300, 512), operands(rng, 200, 1, 300, 512)
    want = [ar.fp8_gemm(o[0], o[1], o[2][0], o[3][0]) for o in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [ar.fp8_gemm(o[0], o[1], o[2][0], o[3][0], stream=s)
               for o, s in zip((a, b), streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def _relative(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


@pytest.mark.parametrize("M", [5, 260])
def test_mlp_of_a_block(M):
    """The MLP half of a decoder block in e4m3, h + W_down·(SiLU(gate)·up) of the
    norm: every operand's codes are within half a step of 2^-4, so each product's
    inputs are off by at most 2^-4 relative and its output, a sum of many terms of
    random sign, by that at most in the 2-norm; three quantized operand pairs
    give 6·2^-4 in the worst case."""
    D, FF = 512, 640
    rng = np.random.default_rng(M)
    X, x = given(rng.standard_normal((M, D)), "bf16")
    Rs, r = given(rng.standard_normal((M, D)), "bf16")
    W, w = given(1 + 0.1 * rng.standard_normal(D), "bf16")
    Wgu, gu = given(rng.standard_normal((2 * FF, D)) / np.sqrt(D), "bf16")
    Wd, d = given(rng.standard_normal((D, FF)) / np.sqrt(FF), "bf16")
    qgu, qd = ar.fp8_quant_weight(Wgu), ar.fp8_quant_weight(Wd)
    n = ar.rmsnorm_fp8(X, W, residual=Rs)
    z = ar.fp8_quant_act(ar.fp8_gemm(n.q, n.scale, *qgu), gate=True)
    out = ar.fp8_gemm(*z, *qd, out_dtype=torch.float32)
    torch.cuda.synchronize()
    y = F.rmsnorm(to_np(n.h).astype(np.float64), w, 1e-6)
    want = F.silu_mul(y @ gu.T) @ d.T
    err = _relative(to_np(out), want)
    log(f"  M={M}: rel err {err:.3f}")
    assert err <= 6 * 2.0 ** -4


def test_experts_of_a_layer():
    """A fused-expert MLP: tokens routed to 2 of 6 experts, gathered by the product
    itself, both products by expert, against the same operators one expert at a time."""
    T, E, D, FF = 90, 6, 256, 384
    rng = np.random.default_rng(8)
    X, _ = given(rng.standard_normal((T, D)), "bf16")
    W, _ = given(np.ones(D), "bf16")
    wgu = ar.fp8_quant_weight(given(0.06 * rng.standard_normal((E, 2 * FF, D)), "bf16")[0])
    wd = ar.fp8_quant_weight(given(0.05 * rng.standard_normal((E, D, FF)), "bf16")[0])
    chosen = np.stack([rng.permutation(E - 1)[:2] for _ in range(T)]).reshape(-1)  # the last: none
    order = np.argsort(chosen, kind="stable")
    off = np.concatenate([[0], np.cumsum(np.bincount(chosen, minlength=E))]).astype(np.int32)
    offd = torch.from_numpy(off).to(dev())
    idx = torch.from_numpy((order // 2).astype(np.int32)).to(dev())
    n = ar.rmsnorm_fp8(X, W)
    y = ar.fp8_gemm_grouped(n.q, n.scale, *wgu, offd, row_index=idx)
    z = ar.fp8_quant_act(y, gate=True)
    out = ar.fp8_gemm_grouped(*z, *wd, offd, out_dtype=torch.float32)
    torch.cuda.synchronize()
    for e in range(E):
        rows = idx[off[e]:off[e + 1]].long()
        if len(rows) == 0:
            continue
        ye = ar.fp8_gemm(n.q.view(torch.uint8)[rows].view(F8), n.scale[:, rows].contiguous(),
                         wgu[0][e], wgu[1][e])
        ze = ar.fp8_quant_act(ye, gate=True)
        one = ar.fp8_gemm(*ze, wd[0][e], wd[1][e], out_dtype=torch.float32)
        torch.cuda.synchronize()
        # the two may sum K in different orders, which can move a code of z by one step
        assert _relative(to_np(out)[off[e]:off[e + 1]], to_np(one)) <= 2.0 ** -4


def test_a_packed_layer_served_in_e4m3():
    """A layer's RTN weight (the codes ar_pack packs) quantized again to e4m3: the
    product stays within the two formats' half steps (2^-4 each operand)."""
    N, K, M = 256, 512, 40
    rng = np.random.default_rng(5)
    Wd, _ = given(0.02 * rng.standard_normal((N, K)), "bf16")
    X, x = given(rng.standard_normal((M, K)), "bf16")
    cfg = ar.Config(bits=8, group_size=128)
    codes, scale, zp, Wq = ar.rtn_quant(Wd, cfg)
    qw, qz = ar.pack(codes, zp, 8)
    a = ar.dequant_gemm(X, qw, qz, scale, 8, 128, N)
    b = ar.fp8_gemm(*ar.fp8_quant_act(X), *ar.fp8_quant_weight(Wq), out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert _relative(to_np(b), to_np(a)) <= 2 * 2.0 ** -4


# ------------------------------------------------------------------ refusals
def test_refusals():
    z = lambda *s, d=torch.float32: torch.zeros(s, dtype=d, device=dev())   # noqa: E731
    M, N, K, E = 8, 144, 256, 3
    KB, NB = 2, 2
    xq, xs, wq, ws = z(M, K, d=F8), z(KB, M), z(N, K, d=F8), z(NB, KB)
    ar.fp8_gemm(xq, xs, wq, ws)
    bad = [(z(M, K), xs, wq, ws), (xq[:, :128], xs, wq, ws), (xq, z(M, KB), wq, ws),
           (xq, z(KB, M, d=BF16), wq, ws), (xq, xs, z(N, K + 16, d=F8), ws),
           (xq, xs, wq, z(NB, KB + 1)), (xq, xs, wq[None], ws), (xq, xs, wq, ws[:1]),
           (xq.cpu(), xs, wq, ws), (None, xs, wq, ws), (xq, xs, wq, None)]
    for args in bad:
        with pytest.raises(ValueError):
            ar.fp8_gemm(*args)
    for kw in (dict(out=z(M, N + 1)), dict(out=z(M, N, d=torch.float16))):
        with pytest.raises(ValueError):
            ar.fp8_gemm(xq, xs, wq, ws, **kw)
    with pytest.raises(TypeError):
        ar.fp8_gemm(xq, xs, wq, ws, out_dtype=torch.float16)
    with pytest.raises(ar.ArError) as e:      # K not a multiple of 16
        ar.fp8_gemm(z(M, 24, d=F8), z(1, M), z(N, 24, d=F8), z(NB, 1))
    assert e.value.status == 3

    off, idx = z(E + 1, d=torch.int32), z(M, d=torch.int32)
    w3, s3 = z(E, N, K, d=F8), z(E, NB, KB)
    ar.fp8_gemm_grouped(xq, xs, w3, s3, off)
    ar.fp8_gemm_grouped(xq, xs, w3, s3, off, row_index=idx)
    for args, kw in (((xq, xs, wq, ws, off), {}), ((xq, xs, w3, s3, off[:-1]), {}),
                     ((xq, xs, w3, s3, off.long()), {}), ((xq, xs, w3, s3, None), {}),
                     ((xq, xs, w3, s3, off), dict(row_index=idx[None])),
                     ((xq, xs, w3, s3, off), dict(row_index=idx.long())),
                     ((xq, xs, w3, s3, off), dict(row_index=idx, out=z(M + 1, N)))):
        with pytest.raises(ValueError):
            ar.fp8_gemm_grouped(*args, **kw)

    for call in (lambda: ar.fp8_quant_act(z(4, 32, d=torch.float16)),
                 lambda: ar.fp8_quant_act(z(32)),
                 lambda: ar.fp8_quant_act(z(4, 65), gate=True),
                 lambda: ar.fp8_quant_act(z(64, 32).t()),
                 lambda: ar.fp8_quant_weight(z(32)),
                 lambda: ar.fp8_quant_weight(z(2, 2, 4, 16)),
                 lambda: ar.rmsnorm_fp8(z(4, 32), z(16)),
                 lambda: ar.rmsnorm_fp8(z(4, 32), z(32, d=BF16)),
                 lambda: ar.rmsnorm_fp8(z(4, 32), z(32), residual=z(4, 16)),
                 lambda: ar.rmsnorm_fp8(z(4, 32), z(32), h_out=z(4, 32))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ar.fp8_quant_act(z(4, 40)), lambda: ar.fp8_quant_weight(z(4, 40)),
                 lambda: ar.rmsnorm_fp8(z(4, 40), z(40))):
        with pytest.raises(ar.ArError):
            call()
    with pytest.raises(ar.ArError):
        ar.rmsnorm_fp8(z(4, 32), z(32), float("nan"))
    torch.cuda.synchronize()
