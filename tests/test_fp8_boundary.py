"""The e4m3 entry points' argument checks on a host without a GPU: every refusal
happens before any HIP call, and the empty problems are no-ops."""
import ctypes

import pytest
import torch

import autoround_signsgd_rounding_amd as ar

pytestmark = pytest.mark.skipif(
    torch.cuda.is_available(),
    reason="validation-only tests pass fake device pointers; they run on a host without a GPU")

OK, INV, UNSUP, SHAPE = 0, 1, 2, 3
P = ctypes.c_void_p(0x100000)          # fake, 16-byte aligned, never dereferenced
P4 = ctypes.c_void_p(0x100004)         # 4-byte aligned
P2 = ctypes.c_void_p(0x100002)
NULL = None


def act(xdt=1, X=P, gate=0, M=4, K=128, q=P, s=P):
    return ar.lib.ar_fp8_quant_act(xdt, X, gate, M, K, q, s, NULL)


def test_quant_act_validation():
    assert act(xdt=2) == UNSUP
    assert act(gate=2) == act(gate=-1) == INV
    for kw in (dict(M=-1), dict(K=-16), dict(K=24), dict(K=1 << 22), dict(M=1 << 23)):
        assert act(**kw) == SHAPE
    for kw in (dict(X=NULL), dict(q=NULL), dict(s=NULL), dict(X=P4), dict(q=P4), dict(s=P2)):
        assert act(**kw) == INV
    assert act(M=0) == act(K=0) == act(M=0, X=NULL) == OK


def weight(wdt=1, W=P, E=1, N=4, K=128, q=P, s=P):
    return ar.lib.ar_fp8_quant_weight(wdt, W, E, N, K, q, s, NULL)


def test_quant_weight_validation():
    assert weight(wdt=9) == UNSUP
    for kw in (dict(E=-1), dict(N=-1), dict(K=8), dict(E=1 << 20, N=128 * 64, K=128 * 64)):
        assert weight(**kw) == SHAPE
    for kw in (dict(W=NULL), dict(q=NULL), dict(s=NULL), dict(W=P4), dict(q=P4), dict(s=P2)):
        assert weight(**kw) == INV
    assert weight(E=0) == weight(N=0) == weight(K=0) == OK


def norm(dt=1, x=P, r=P, w=P, M=4, D=128, eps=1e-6, h=P, y=P, q=P, s=P):
    return ar.lib.ar_rmsnorm_fp8(dt, x, r, w, M, D, eps, h, y, q, s, NULL)


def test_rmsnorm_validation():
    assert norm(dt=5) == UNSUP
    for eps in (-1e-6, float("nan"), float("inf")):
        assert norm(eps=eps) == INV
    for kw in (dict(M=-1), dict(D=136), dict(D=-16), dict(M=1 << 23)):
        assert norm(**kw) == SHAPE
    for kw in (dict(x=NULL), dict(w=NULL), dict(q=NULL), dict(s=NULL), dict(r=NULL), dict(x=P4),
               dict(r=P4), dict(w=P4), dict(h=P4), dict(y=P4), dict(q=P4), dict(s=P2)):
        assert norm(**kw) == INV             # h without a residual among them
    assert norm(M=0) == norm(D=0) == OK


def gemm(X=P, xs=P, M=4, K=128, W=P, ws=P, N=64, Y=P, ydt=1):
    return ar.lib.ar_fp8_gemm(X, xs, M, K, W, ws, N, Y, ydt, NULL)


def grouped(X=P, xs=P, T=4, K=128, W=P, ws=P, E=2, N=64, off=P, idx=NULL, R=4, Y=P, ydt=1):
    return ar.lib.ar_fp8_gemm_grouped(X, xs, T, K, W, ws, E, N, off, idx, R, Y, ydt, NULL)


@pytest.mark.parametrize("f", [gemm, grouped])
def test_product_validation(f):
    assert f(ydt=2) == UNSUP
    for kw in (dict(K=0), dict(K=120), dict(K=-16), dict(N=-1), dict(K=1 << 22), dict(N=1 << 23)):
        assert f(**kw) == SHAPE
    for kw in (dict(X=NULL), dict(xs=NULL), dict(W=NULL), dict(ws=NULL), dict(Y=NULL), dict(X=P4),
               dict(W=P4), dict(Y=P4), dict(xs=P2), dict(ws=P2)):
        assert f(**kw) == INV
    assert f(N=0) == OK
    # the scales may start at any float
    assert f(xs=P4, ws=P4, Y=NULL) == INV and f(xs=P4, ws=P4, N=0) == OK


def test_gemm_rows():
    assert gemm(M=-1) == gemm(M=1 << 23) == SHAPE
    assert gemm(M=0) == OK


def test_grouped_validation():
    for kw in (dict(E=0), dict(E=8193), dict(R=5), dict(T=-1, R=-1), dict(T=0, idx=P, R=4),
               dict(T=1 << 22, K=1024, idx=P, R=8), dict(R=1 << 23, T=1 << 23)):
        assert grouped(**kw) == SHAPE
    for kw in (dict(off=NULL), dict(off=P2), dict(idx=P2)):
        assert grouped(**kw) == INV
    assert grouped(T=0, R=0) == grouped(T=9, idx=P, R=0) == OK



@pytest.mark.parametrize("f", [gemm, grouped])
def test_sums_flag_validation(f):
    """AR_F32_SUMS goes with either output type; other bits are refused."""
    for ydt in (0, 1, 0x100, 0x101):
        assert f(ydt=ydt, N=0) == OK and f(ydt=ydt, Y=NULL) == INV
    for ydt in (2, 0x102, 0x200, 0x201, 0x301, -1, -256):
        assert f(ydt=ydt) == f(ydt=ydt, N=0) == UNSUP
