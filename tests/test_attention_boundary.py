"""The attention and 4-bit cache entry points' argument checks on a host without a GPU: every
refusal happens before any HIP call, and the empty problems are no-ops."""
import ctypes

import pytest
import torch

import autoround_signsgd_rounding_amd as ar

pytestmark = pytest.mark.skipif(
    torch.cuda.is_available(),
    reason="validation-only tests pass fake device pointers; they run on a host without a GPU")

OK, INV, UNSUP, SHAPE, WS = 0, 1, 2, 3, 4
P = ctypes.c_void_p(0x100000)          # fake, 16-byte aligned, never dereferenced
P4 = ctypes.c_void_p(0x100004)
P2 = ctypes.c_void_p(0x100002)
NULL = None
NAN, INF = float("nan"), float("inf")


def cache(**kw):
    a = dict(codes=0x100000, scale=0x100000, pages=8, heads=2, head_dim=128, page_size=64,
             group_size=128)
    a.update(kw)
    return ctypes.byref(ar.ArKv4Cache(*a.values()))


BAD_CACHES = [(dict(head_dim=96), UNSUP), (dict(head_dim=256), UNSUP), (dict(group_size=16), UNSUP),
              (dict(group_size=-1), UNSUP), (dict(group_size=128, head_dim=64), UNSUP),
              (dict(page_size=8), UNSUP), (dict(page_size=48), UNSUP), (dict(page_size=512), UNSUP),
              (dict(page_size=-16), UNSUP), (dict(pages=0), SHAPE), (dict(pages=1 << 25), SHAPE),
              (dict(heads=0), SHAPE), (dict(heads=1 << 16), SHAPE)]
BAD_ARRAYS = [dict(codes=0), dict(scale=0), dict(codes=0x100004), dict(scale=0x100004)]


def write(c=None, dt=1, k=P, ks=256, v=P, vs=256, slots=P, T=4):
    return ar.lib.ar_kv4_write(cache() if c is None else c, dt, k, ks, v, vs, slots, T, NULL)


def read(c=None, slots=P, T=4, dt=1, k=P, v=P):
    return ar.lib.ar_kv4_read(cache() if c is None else c, slots, T, dt, k, v, NULL)


@pytest.mark.parametrize("f", [write, read])
def test_cache_validation(f):
    for kw, want in BAD_CACHES:
        assert f(c=cache(**kw)) == f(c=cache(**kw), T=0) == want, kw
    for kw in BAD_ARRAYS:
        assert f(c=cache(**kw)) == INV, kw
    assert f(c=ctypes.POINTER(ar.ArKv4Cache)()) == INV
    assert f(dt=2) == UNSUP
    assert f(T=-1) == f(T=1 << 31) == f(T=1 << 28) == SHAPE     # (a launch holds 2^32 threads)
    for kw in (dict(k=NULL), dict(v=NULL), dict(slots=NULL), dict(k=P4), dict(v=P4), dict(slots=P2)):
        assert f(**kw) == INV
    assert f(T=0) == f(T=0, k=NULL, v=NULL, slots=NULL) == OK


def test_write_strides():
    for s in (255, 248, 260, -256, 1 << 22):
        assert write(ks=s) == write(vs=s) == SHAPE
    assert write(ks=264, vs=1024, k=NULL) == INV      # the strides are fine


def attention(c=None, q=P, qs=1024, B=2, n=1, H=8, table=P, width=4, lengths=P, max_len=256,
              scale=0.1, out=P, lse=P, ws=P, size=1 << 40):
    return ar.lib.ar_kv4_attention(cache() if c is None else c, q, qs, B, n, H, table, width,
                                   lengths, max_len, scale, out, lse, ws, size, NULL)


def test_kv4_attention_validation():
    for kw, want in BAD_CACHES:
        assert attention(c=cache(**kw)) in (want, SHAPE), kw
    for kw in BAD_ARRAYS:
        assert attention(c=cache(**kw)) == INV, kw
    for kw in (dict(H=7), dict(H=0), dict(H=1024, qs=1024 * 128), dict(n=-1), dict(n=257),
               dict(B=-1), dict(B=1 << 31), dict(B=1 << 28), dict(B=1 << 22), dict(max_len=-1), dict(max_len=257),
               dict(width=1 << 25), dict(width=-1), dict(qs=1016), dict(qs=1028),
               dict(max_len=1 << 30, width=1 << 24)):
        assert attention(**kw) == SHAPE, kw
    for kw in (dict(q=NULL), dict(table=NULL), dict(lengths=NULL), dict(out=NULL), dict(q=P4),
               dict(out=P4), dict(table=P2), dict(lengths=P2), dict(lse=P2), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=NAN), dict(scale=INF)):
        assert attention(**kw) == INV, kw
    assert attention(B=0) == attention(n=0) == OK


def size_of(**kw):
    a = dict(B=2, n=1, H=8, max_len=1 << 20)
    a.update(kw)
    out = ctypes.c_size_t(77)
    st = ar.lib.ar_kv4_attention_workspace_size(cache(), *a.values(), ctypes.byref(out))
    return st, out.value


def test_kv4_workspace():
    st, need = size_of()
    assert st == OK and need > 0
    assert attention(max_len=1 << 20, width=1 << 14, size=need - 1) == WS
    assert attention(max_len=1 << 20, width=1 << 14, size=need, ws=NULL) == INV
    assert attention(max_len=1 << 20, width=1 << 14, size=need, ws=P4) == INV
    assert size_of(max_len=0) == size_of(B=0) == (OK, 0)
    assert size_of(H=7)[0] == SHAPE
    assert ar.lib.ar_kv4_attention_workspace_size(cache(), 2, 1, 8, 64, None) == INV


def packed(q=P, qs=1024, k=P, ks=256, v=P, vs=256, Tq=4, Tk=4, H=8, Hk=2, D=128, qo=P, ko=NULL,
           B=1, scale=0.1, out=P, lse=NULL, ws=NULL, size=0):
    return ar.lib.ar_attention_packed(q, qs, k, ks, v, vs, Tq, Tk, H, Hk, D, qo, ko, B, scale, out,
                                      lse, ws, size, NULL)


def test_packed_validation():
    assert packed(D=96, qs=768) == packed(D=256, qs=2048) == UNSUP
    for kw in (dict(H=7), dict(Hk=0), dict(H=0), dict(H=1024, qs=1024 * 128), dict(B=-1),
               dict(B=65537), dict(Tq=-1), dict(Tk=-1), dict(Tk=5), dict(Tq=1 << 31),
               dict(Tq=1 << 28, Tk=1 << 28), dict(Tk=1 << 30, ko=P), dict(qs=1016), dict(ks=252), dict(vs=128),
               dict(ks=1 << 22), dict(Tq=1 << 27, Tk=1 << 27),
               dict(B=65536, Tq=65536, Tk=65536, H=64, Hk=64, qs=8192, ks=8192, vs=8192)):
        assert packed(**kw) == SHAPE, kw
    for kw in (dict(q=NULL), dict(k=NULL), dict(v=NULL), dict(qo=NULL), dict(out=NULL), dict(q=P4),
               dict(k=P4), dict(v=P4), dict(out=P4), dict(qo=P2), dict(ko=P2), dict(lse=P2),
               dict(scale=0.0), dict(scale=NAN), dict(scale=INF), dict(scale=-0.1)):
        assert packed(**kw) == INV, kw
    assert packed(Tq=0, Tk=0) == packed(B=0) == packed(Tq=0, ko=P) == OK


def test_packed_workspace():
    out = ctypes.c_size_t(5)
    f = ar.lib.ar_attention_packed_workspace_size
    assert f(1, 4, 4, 8, 2, 128, ctypes.byref(out)) == OK
    assert f(1, 4, 4, 8, 3, 128, ctypes.byref(out)) == SHAPE
    assert f(1, 4, 4, 8, 2, 32, ctypes.byref(out)) == UNSUP
    assert f(1, 4, 4, 8, 2, 128, None) == INV


def test_binding_refuses_on_the_host():
    """Tensors of the CPU, and cache shapes that contradict themselves, raise ValueError."""
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    kv = (torch.zeros((8, 2, 2, 64, 64), dtype=torch.uint8), torch.zeros((8, 2, 2, 64, 1)))
    with pytest.raises(ValueError):
        ar.attention_packed(x, x, x, i)
    for bad in (None, (None, None), kv, kv[:1], (kv[0][0], kv[1]), (kv[0], kv[1][..., :0])):
        with pytest.raises(ValueError):
            ar.kv4_write(x, x, bad, i)
        with pytest.raises(ValueError):
            ar.kv4_read(bad, i)
        with pytest.raises(ValueError):
            ar.kv4_attention(x, bad, i[None], i)
    for kw in (dict(page_size=8), dict(page_size=24), dict(group_size=16), dict(group_size=256),
               dict(pages=0), dict(heads=0), dict(head_dim=96)):
        with pytest.raises(ValueError):
            ar.kv4_cache(**{**dict(pages=4, heads=2, head_dim=128, device="cpu"), **kw})
    assert ar.kv4_cache(4, 2, 64, page_size=16, group_size=32, device="cpu").scale.shape == \
        (4, 2, 2, 16, 2)


def test_scales_whose_logarithm_leaves_float32():
    """scale·log2(e) is what the kernels multiply by: it has to be a float32."""
    for s in (2.4e38, 3.4028e38):
        assert packed(scale=s) == attention(scale=s) == INV
    most = 2.3e38
    assert packed(Tk=4000, ko=P, scale=most) == WS
    assert attention(max_len=1 << 20, width=1 << 14, size=0, scale=most) == WS


@pytest.mark.parametrize("f", [write, read])
def test_tokens_of_one_launch(f):
    """16 tokens a workgroup of 256 threads: 2^24 workgroups are a thread more than a launch holds."""
    most = ((1 << 24) - 1) * 16
    assert f(T=most + 1) == f(T=(1 << 28) - 1) == SHAPE
    assert f(T=most, k=NULL) == INV     # the size is fine


def test_packed_f32_validation():
    """The form with float32 weights refuses what the other does."""
    def f(**kw):
        a = dict(q=P, qs=1024, k=P, ks=256, v=P, vs=256, Tq=4, Tk=4, H=8, Hk=2, D=128, qo=P, ko=NULL,
                 B=1, scale=0.1, out=P, lse=NULL, ws=NULL, size=0)
        a.update(kw)
        return ar.lib.ar_attention_packed_f32(*a.values(), NULL)
    assert f(D=96, qs=768) == UNSUP
    assert f(H=7) == f(Tk=5) == f(qs=1016) == f(ks=252) == f(B=65537) == SHAPE
    assert f(q=NULL) == f(v=P4) == f(out=NULL) == f(scale=0.0) == f(qo=P2) == INV
    assert f(Tk=4000, ko=P) == WS
    assert f(Tq=0, Tk=0) == f(B=0) == OK
