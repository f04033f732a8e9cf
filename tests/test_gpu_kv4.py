"""The 4-bit cache: written and read back against the oracle bit for bit; attention over it
against the oracle in float64 on the values that it holds."""
import numpy as np
import pytest
import torch

from attention_common import bf16, check, i32, keys, lse_bound, out_bound
from gpu_common import dev, log
from oracle import kv4_ref as R

pytestmark = pytest.mark.gpu
ar = pytest.importorskip("autoround_signsgd_rounding_amd")

W_BITS = 2.0 ** -11      # weights are rounded to f16
F32 = np.float32


def arrays(pages, heads, D, P, group, fill=0xA5):
    return (np.full((pages, 2, heads, P, D // 2), fill, np.uint8),
            np.full((pages, 2, heads, P, D // group), 3.5, F32))


def on_gpu(cache):
    return ar.KV4Cache(*(torch.from_numpy(x).to(dev()) for x in cache))


def same(got, want):
    assert np.array_equal(got[0].cpu().numpy(), want[0])
    assert np.array_equal(got[1].cpu().numpy().view(np.uint32), want[1].view(np.uint32))


# ------------------------------------------------------------------ written and read
SHAPES = [(1, 1, 64, 16, 64), (5, 2, 128, 32, 128), (77, 3, 64, 16, 32), (300, 2, 128, 64, 64),
          (130, 1, 128, 128, 32), (33, 5, 64, 256, 32), (600, 8, 128, 64, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,heads,D,P,group", SHAPES)
def test_write_and_read(T, heads, D, P, group, dtype):
    """Codes and scales bit for bit, everything else as it was; values read back exactly."""
    log(f"kv4 write {T} x {heads} x {D} page {P} group {group} {dtype}")
    rng = np.random.default_rng(T)
    pages = -(-T // P) + 2
    k, v = keys(rng, T, heads, D).astype(F32), rng.normal(size=(T, heads, D)).astype(F32)
    slots = rng.permutation(pages * P)[:T].astype(np.int32)
    if T > 4:
        slots[1], slots[3], slots[4] = -1, pages * P, -(1 << 31)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    K, V = (torch.from_numpy(x).to(dev()).to(dt) for x in (k, v))
    want = arrays(pages, heads, D, P, group)
    cache = on_gpu(want)
    R.write(*want, K.float().cpu().numpy(), V.float().cpu().numpy(), slots)
    assert ar.kv4_write(K, V, cache, i32(slots)) is None
    same(cache, want)
    for out in (torch.float32, torch.bfloat16):
        for x, w in zip(ar.kv4_read(cache, i32(slots), out_dtype=out), R.held(*want, slots)):
            assert x.dtype is out
            assert torch.equal(x.cpu(), torch.from_numpy(w.astype(F32)).to(out))
    # a slot may be read any number of times
    twice = np.concatenate([slots[:2], slots[:2], slots[-1:]])
    for x, w in zip(ar.kv4_read(cache, i32(twice), out_dtype=torch.float32), R.held(*want, twice)):
        assert np.array_equal(x.cpu().numpy(), w.astype(F32))


def test_grid_edges():
    """Groups of zeros, of one sign, of one value, tiny, huge, halfway between codes, with NaN
    and infinities."""
    log("kv4 grid edges")
    rows = []
    add = lambda x: rows.append(np.resize(np.asarray(x, F32), 64))      # noqa: E731
    for x in ([0.0], [-0.0], [1.0], [-2.5], [0.0, 15.0], [-15.0, 0.0], np.arange(16) - 7.0,
              np.arange(32) / 2.0 - 7.5, [-1.0, 1.0], [1e-45], [1e-38, -1e-38], [2e-30, 1e-31],
              [3.4e38], [1.7e38, -1.7e38], [3e38, -3e38], [np.nan], [1.0, np.nan], [np.inf, 1.0],
              [-np.inf, 1.0], [np.inf, -np.inf], [2.0 ** -100, 2.0 ** -96], [1e-3, 1e3]):
        add(x)
    rng = np.random.default_rng(0)
    for e in rng.uniform(-30, 37, 200):
        add(rng.normal(size=64) * 10.0 ** e)
    for s in 2.0 ** rng.integers(-90, 90, 200) * rng.integers(1, 1 << 20, 200):
        add((rng.integers(0, 31, 64) / 2.0 - 7.5) * s)                  # halves of a step
    x = np.stack(rows)[:, None]
    want = arrays(len(x) // 16 + 1, 1, 64, 16, 32)
    cache = on_gpu(want)
    slots = np.arange(len(x), dtype=np.int32)
    R.write(*want, x, x[::-1], slots)
    X = torch.from_numpy(x).to(dev())
    ar.kv4_write(X, X.flip(0).contiguous(), cache, i32(slots))
    assert np.array_equal(cache.codes.cpu().numpy(), want[0])
    a, b = cache.scale.cpu().numpy(), want[1]
    assert np.array_equal(np.isnan(a), np.isnan(b))
    assert np.array_equal(a[~np.isnan(a)].view(np.uint32), b[~np.isnan(b)].view(np.uint32))


def test_strided_tokens_and_repeated_slots():
    """Parts of one product; a slot named twice spoils itself only."""
    log("kv4 strided")
    rng = np.random.default_rng(2)
    T, heads, D, P = 40, 2, 64, 16
    qkv = torch.from_numpy(rng.normal(size=(T, 8, D)).astype(F32)).to(dev())
    K, V = qkv[:, 4:6], qkv[:, 6:]
    want = arrays(3, heads, D, P, 32)
    cache = on_gpu(want)
    slots = rng.permutation(48)[:T].astype(np.int32)
    slots[9] = slots[7]
    R.write(*want, K.cpu().numpy(), V.cpu().numpy(), slots)
    ar.kv4_write(K, V, cache, i32(slots))
    got = ar.kv4_read(cache, i32([s for s in range(48) if s != slots[7]]), out_dtype=torch.float32)
    held = R.held(*want, [s for s in range(48) if s != slots[7]])
    for g, w in zip(got, held):
        assert np.array_equal(g.cpu().numpy(), w.astype(F32))


def test_far_pages():
    """A cache beyond 4 GiB: offsets of its last pages pass 32 bits."""
    log("kv4 far pages")
    pages, heads, D, P = 70000, 8, 128, 64
    cache = ar.kv4_cache(pages, heads, D, page_size=P)
    assert cache.codes.numel() > 1 << 32
    rng = np.random.default_rng(1)
    T = 100
    (K, k), (V, v) = bf16(rng.normal(size=(T, heads, D))), bf16(rng.normal(size=(T, heads, D)))
    last = pages * P - 1
    slots = np.arange(last, last - T, -1)
    ar.kv4_write(K, V, cache, i32(slots))
    for g, x in zip(ar.kv4_read(cache, i32(slots), out_dtype=torch.float32), (k, v)):
        c, s = R.grid(x, D)
        w = (c - (s.view(np.uint32) & 15).astype(float)) * s
        assert np.array_equal(g.cpu().numpy(), w.astype(F32))
    # the sequence's tokens in order are those of the last pages backwards, token by token
    order = slots.reshape(-1)[::-1] // P
    table = i32(np.unique(order)[None])
    n = int(last - np.unique(order)[0] * P + 1)
    q, qv = bf16(rng.normal(size=(1, 8, D)))
    got = ar.kv4_attention(q, cache, table, i32([n]), want_lse=True)
    first = np.unique(order)[0] * P
    kk, vv = (x.double().cpu().numpy() for x in
              ar.kv4_read(cache, i32(np.arange(first, last + 1)), out_dtype=torch.float32))
    compare(got, qv[:, None], [kk], [vv], 1, "far")
    del cache
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ attention
def compare(got, q, ks, vs, new, what, scale=None, gone=None):
    """kv4_attention's outputs against the oracle's: q [B, new, H, D]; ks, vs [n, heads, D] of
    each sequence; gone: keys of each sequence that take no part."""
    B, _, H, D = q.shape
    out, lse = got.out.double().cpu().numpy().reshape(q.shape), got.lse.cpu().numpy().reshape(B, new, H)
    for b in range(B):
        n, r = len(ks[b]), H // ks[b].shape[1]
        sees = R.causal(new, n)
        if gone is not None:
            sees = sees & ~gone[b][None]
        for h in range(H):
            o, l, size, mag = R.rows(q[b, :, h], ks[b][:, h // r], vs[b][:, h // r], sees,
                                     D ** -0.5 if scale is None else scale)
            empty = np.isneginf(l)
            assert (np.isneginf(lse[b, :, h]) == empty).all() and (out[b, empty, h] == 0).all()
            if n == 0:
                continue
            # what the matrix unit cuts off, with scales of a token's keys or values of at most a
            # seventh of their largest: of a score, 2^-17 of scale times max |q| a channel; of
            # a value's product and its zero-point's, 2^-14 of the largest of 8 weights each
            ktop = np.abs(ks[b][:, h // r]).max(1) / 7
            vtop = np.abs(vs[b][:, h // r]).max(1) / 7
            sc = D ** -0.5 if scale is None else scale
            cut = D * 2.0 ** -17 * np.abs(q[b, :, h]).max(1) * sc * ktop.max()
            weight = np.stack([R.rows(q[b, i:i + 1, h], ks[b][:, h // r], vtop[:, None],
                                      sees[i:i + 1], sc)[0][0] for i in range(new)])
            # weights below 2^-30 of the largest may vanish
            bound = out_bound(o, size, mag, D, n, W_BITS) + size * 2 * np.expm1(cut)[:, None] + \
                2.0 ** -10 * weight + n * 2.0 ** -30 * 8 * vtop.max()
            check(out[b, :, h], o, bound, f"{what}: out {b} {h}")
            bound = lse_bound(l, mag, D, n) + cut
            check(lse[b, ~empty, h], l[~empty], bound[~empty], f"{what}: lse {b} {h}")


def filled(rng, lengths, heads, D, P, group, spare=2):
    """A cache in which the sequences' pages lie anywhere, every other place holding NaN
    scales, and what it holds for each."""
    per = [-(-n // P) for n in lengths]
    pages = sum(per) + spare
    order = rng.permutation(pages)
    width = max(max(per), 1) + 1
    table = np.full((len(lengths), width), -1, np.int32)
    cache = ar.kv4_cache(pages, heads, D, page_size=P, group_size=group, device=dev())
    cache.codes.fill_(0x3C)
    cache.scale.fill_(float("nan"))
    ks, vs, at = [], [], 0
    for b, n in enumerate(lengths):
        mine = order[at:at + per[b]]
        at += per[b]
        table[b, :per[b]] = mine
        t = np.arange(n)
        slots = mine[t // P] * P + t % P if n else np.zeros(0, int)
        K, V = bf16(keys(rng, n, heads, D))[0], bf16(rng.normal(size=(n, heads, D)))[0]
        ar.kv4_write(K, V, cache, i32(slots))
        k, v = ar.kv4_read(cache, i32(slots), out_dtype=torch.float32)
        ks.append(k.double().cpu().numpy())
        vs.append(v.double().cpu().numpy())
    return cache, i32(table), ks, vs


CASES = [  # lengths, new, heads, key heads, head_dim, page, group
    ([1], 1, 1, 1, 64, 16, 64),
    ([1, 15, 16, 17, 31, 32, 33], 1, 4, 2, 128, 16, 128),
    ([100], 1, 8, 8, 128, 64, 128),
    ([129, 500, 7], 1, 16, 2, 64, 32, 32),
    ([1000], 1, 8, 1, 128, 128, 64),
    ([257, 1300], 1, 6, 2, 128, 16, 32),
    ([90, 40], 5, 14, 2, 64, 16, 32),
    ([300, 3, 65], 4, 8, 1, 128, 64, 128),          # 32 rows; a sequence shorter than the draft
    ([600], 8, 8, 1, 128, 32, 64),                  # 64 rows
    ([77, 0, 5], 1, 4, 1, 64, 16, 64),              # a sequence without tokens
    ([2, 0], 3, 2, 2, 128, 64, 32),
    ([50], 1, 256, 1, 64, 16, 32),                  # the largest group
    ([260], 3, 17, 1, 128, 256, 128),
    ([40, 300], 256, 2, 1, 64, 32, 64),             # the most new tokens, more than there are
    ([20], 2, 300, 300, 64, 16, 32),                # many key heads
]


@pytest.mark.parametrize("lengths,new,H,heads,D,P,group", CASES)
def test_attention(lengths, new, H, heads, D, P, group):
    log(f"kv4 attention {lengths} new {new} heads {H}/{heads} x {D} page {P} group {group}")
    rng = np.random.default_rng(sum(lengths) + H)
    cache, table, ks, vs = filled(rng, lengths, heads, D, P, group)
    Q, q = bf16(1.5 * rng.normal(size=(len(lengths), new, H, D)))
    got = ar.kv4_attention(Q, cache, table, i32(lengths), want_lse=True)
    torch.cuda.synchronize()
    compare(got, q, ks, vs, new, "kv4")
    bare = ar.kv4_attention(Q, cache, table, i32(lengths))
    assert bare.lse is None and torch.equal(bare.out, got.out)
    if new == 1:
        flat = ar.kv4_attention(Q[:, 0], cache, table, i32(lengths))
        assert flat.out.shape == (len(lengths), H, D) and torch.equal(flat.out, got.out[:, 0])


@pytest.mark.parametrize("H,heads,new,group", [(8, 1, 1, 128), (32, 8, 1, 64), (4, 2, 3, 32)])
def test_long_sequences(H, heads, new, group):
    """Several workgroups share a sequence; neighbours are short."""
    log(f"kv4 long {H}/{heads} new {new} group {group}")
    rng = np.random.default_rng(H)
    lengths = [9001, 3, 4096, 700]
    cache, table, ks, vs = filled(rng, lengths, heads, 128, 64, group)
    Q, q = bf16(1.5 * rng.normal(size=(4, new, H, 128)))
    got = ar.kv4_attention(Q, cache, table, i32(lengths), want_lse=True)
    compare(got, q, ks, vs, new, "long")
    # a bound on the lengths divides the work otherwise; a longer one is cut to it
    tight = ar.kv4_attention(Q, cache, table, i32(lengths), max_len=9001, want_lse=True)
    compare(tight, q, ks, vs, new, "bounded")
    cut = ar.kv4_attention(Q, cache, table, i32(lengths), max_len=1000, want_lse=True)
    compare(cut, q, [k[:1000] for k in ks], [v[:1000] for v in vs], new, "cut")


@pytest.mark.parametrize("lengths,new,H,heads,D,P,group", [
    ([300, 3, 65], 4, 8, 1, 128, 64, 128), ([600], 8, 8, 1, 128, 32, 64), ([90, 2000], 5, 14, 2, 64, 16, 32),
    ([1500, 700, 5], 3, 24, 3, 64, 128, 64), ([700], 17, 4, 2, 128, 16, 32)])
def test_room_for_long_sequences(lengths, new, H, heads, D, P, group):
    """Many rows a key head, under a table that has room for a great deal more."""
    log(f"kv4 room {lengths} new {new} heads {H}/{heads} x {D} page {P} group {group}")
    rng = np.random.default_rng(sum(lengths))
    cache, table, ks, vs = filled(rng, lengths, heads, D, P, group)
    width = -(-400000 // (len(lengths) * heads * P))
    wide = torch.full((len(lengths), width), -1, dtype=torch.int32, device=dev())
    wide[:, :table.shape[1]] = table
    Q, q = bf16(1.5 * rng.normal(size=(len(lengths), new, H, D)))
    got = ar.kv4_attention(Q, cache, wide, i32(lengths), want_lse=True)
    compare(got, q, ks, vs, new, "room")


@pytest.mark.parametrize("new", [1, 3])
def test_many_short_sequences(new):
    """More sequences than a wave has lanes, 8 query heads a key head."""
    log(f"kv4 many short sequences, new {new}")
    rng = np.random.default_rng(31)
    lengths = [int(x) for x in rng.integers(0, 40, 400)]
    lengths[350] = 230
    cache, table, ks, vs = filled(rng, lengths, 4, 64, 16, 64)
    Q, q = bf16(1.5 * rng.normal(size=(400, new, 32, 64)))
    got = ar.kv4_attention(Q, cache, table, i32(lengths), want_lse=True)
    compare(got, q, ks, vs, new, "many")


@pytest.mark.parametrize("B", [100, 300])
def test_a_few_long_sequences_among_many(B):
    """More sequences than a wave has lanes, and than it keeps lengths of, some of them divided."""
    log(f"kv4 few long among {B}")
    rng = np.random.default_rng(B)
    lengths = [int(x) for x in rng.integers(0, 40, B)]
    lengths[5], lengths[70], lengths[B - 1] = 1100, 2500, 2200
    cache, table, ks, vs = filled(rng, lengths, 1, 64, 16, 64)
    Q, q = bf16(1.5 * rng.normal(size=(B, 2, 4, 64)))
    got = ar.kv4_attention(Q, cache, table, i32(lengths), want_lse=True)
    compare(got, q, ks, vs, 2, "few long")


def test_strided_queries():
    """Queries [B, n] within a larger array, all of whose tokens lie one stride apart; what
    does not is refused."""
    log("kv4 strided queries")
    rng = np.random.default_rng(32)
    cache, table, ks, vs = filled(rng, [50, 20], 2, 64, 32, 64)
    n = i32([50, 20])
    X, x = bf16(rng.normal(size=(2, 3, 8, 64)))
    got = ar.kv4_attention(X[:, :, 2:6], cache, table, n, want_lse=True)
    assert got.out.is_contiguous()
    compare(got, x[:, :, 2:6], ks, vs, 3, "strided")
    got = ar.kv4_attention(X[:, 1:2, 2:6], cache, table, n, want_lse=True)
    compare(got, x[:, 1:2, 2:6], ks, vs, 1, "one of three")
    got = ar.kv4_attention(X[1:, 1:, 2:6], cache, table[1:], n[1:], want_lse=True)
    compare(got, x[1:, 1:, 2:6], ks[1:], vs[1:], 2, "one sequence")
    with pytest.raises(ValueError, match="one stride apart"):
        ar.kv4_attention(X[:, 1:, 2:6], cache, table, n)


def test_pages_that_are_not_there():
    """Pages outside the cache take no part: -1, beyond it, all of a sequence's."""
    log("kv4 pages that are not there")
    rng = np.random.default_rng(4)
    for P in (16, 32):
        lengths, H, heads, D = [300, 200, 90], 4, 2, 64
        cache, table, ks, vs = filled(rng, lengths, heads, D, P, 32)
        table[0, 3], table[0, 4], table[0, 0] = -1, cache.codes.shape[0], 1 << 30
        table[2] = -(1 << 31)
        gone = [np.isin(np.arange(300) // P, [0, 3, 4]), np.zeros(200, bool), np.ones(90, bool)]
        Q, q = bf16(rng.normal(size=(3, 2, H, D)))
        got = ar.kv4_attention(Q, cache, table, i32(lengths), want_lse=True)
        compare(got, q, ks, vs, 2, f"gone {P}", gone=gone)
        # lengths outside the table
        Q1 = Q[:, :1]
        a = ar.kv4_attention(Q1, cache, table, i32([-5, 1 << 30, -(1 << 31)]), want_lse=True)
        assert (a.out[0] == 0).all() and torch.isneginf(a.lse[0]).all()
        n = table.shape[1] * P
        there = table[1].cpu().numpy()[np.arange(n) // P] >= 0
        if there[200:].any():       # the tail of its last page holds NaN
            assert torch.isnan(a.out[1]).all()


def test_hidden_nan_and_seen_nan():
    """A cached NaN makes the rows that see it NaN; the draft's earlier rows do not see it."""
    log("kv4 nan")
    rng = np.random.default_rng(6)
    H, heads, D, P, n = 4, 2, 128, 16, 70
    cache, table, ks, vs = filled(rng, [n], heads, D, P, 64)
    slot = int(table[0, (n - 1) // P]) * P + (n - 1) % P
    K = torch.ones((1, heads, D), device=dev())
    for which in (0, 1):
        kv = [K.clone(), K.clone()]
        kv[which][0, 1, 70] = float("nan")
        ar.kv4_write(*kv, cache, i32([slot]))
        Q, q = bf16(rng.normal(size=(1, 3, H, D)))
        got = ar.kv4_attention(Q, cache, table, i32([n]), want_lse=True)
        assert torch.isfinite(got.out[0, :2]).all() and torch.isfinite(got.out[0, 2, :2]).all()
        hit = got.out[0, 2, 2:]
        assert torch.isnan(hit[..., 64:]).all()
        assert torch.isnan(hit[..., :64]).all() == (which == 0)


def test_extremes():
    """Queries and values at the ends of bf16's range, sharp and flat rows, tiny values."""
    log("kv4 extremes")
    rng = np.random.default_rng(8)
    H, heads, D, P, n = 8, 2, 64, 32, 150
    for qs, ks_, vs_ in ((1e30, 1e-30, 1e30), (1e-36, 1.0, 1e-25), (40.0, 4.0, 1e-6), (0.0, 1.0, 1e6)):
        cache = ar.kv4_cache(8, heads, D, page_size=P, group_size=32)
        slots = i32(np.arange(n))
        K, V = bf16(ks_ * keys(rng, n, heads, D))[0], bf16(vs_ * rng.normal(size=(n, heads, D)))[0]
        V[5] *= 100
        ar.kv4_write(K, V, cache, slots)
        k, v = (x.double().cpu().numpy() for x in ar.kv4_read(cache, slots, out_dtype=torch.float32))
        Q, q = bf16(qs * rng.normal(size=(1, 1, H, D)))
        got = ar.kv4_attention(Q, cache, i32(np.arange(8)[None]), i32([n]), want_lse=True)
        compare(got, q, [k], [v], 1, f"extremes {qs}")
        got = ar.kv4_attention(Q, cache, i32(np.arange(8)[None]), i32([n]), want_lse=True, scale=0.02)
        compare(got, q, [k], [v], 1, f"extremes {qs}, scale", scale=0.02)


def test_given_outputs_and_workspace():
    log("kv4 given outputs")
    rng = np.random.default_rng(3)
    cache, table, ks, vs = filled(rng, [3000, 50], 2, 128, 64, 128)
    qkv, x = bf16(rng.normal(size=(2, 12, 128)))      # q beside k and v
    Q, out = qkv[:, :8], torch.empty((2, 8, 128), dtype=torch.bfloat16, device=dev())
    ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device=dev())     # NaN all over
    got = ar.kv4_attention(Q, cache, table, i32([3000, 50]), out=out, workspace=ws, want_lse=True)
    assert got.out is out
    compare(got, x[:, None, :8], ks, vs, 1, "given")
    with pytest.raises(ar.ArError, match="WORKSPACE"):
        ar.kv4_attention(Q, cache, table, i32([3000, 50]), workspace=ws[:1024])


def test_binding_checks():
    cache = ar.kv4_cache(4, 2, 64, page_size=16, group_size=32)
    K, s = torch.zeros((5, 2, 64), dtype=torch.bfloat16, device=dev()), i32(range(5))
    ar.kv4_write(K, K, cache, s)
    for a in ((K[..., :32], K, s), (K, K.float(), s), (K, K[:4], s), (K, K, s.long()), (K, K, s[:3]),
              (K, K, s.cpu()), (K.half(), K.half(), s), (K[:, :1], K[:, :1], s), (None, K, s)):
        with pytest.raises(ValueError):
            ar.kv4_write(a[0], a[1], cache, a[2])
    for bad in ((cache.codes, cache.scale[:2]), (cache.codes.int(), cache.scale),
                (cache.codes, cache.scale.double()), (cache.codes, cache.scale.cpu()),
                (cache.codes[:, :, :1], cache.scale[:, :, :1]), (cache.codes[:, :1], cache.scale[:, :1])):
        with pytest.raises(ValueError):
            ar.kv4_read(bad, s)
    with pytest.raises(TypeError):
        ar.kv4_read(cache, s, out_dtype=torch.float16)
    Q, t, n = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device=dev()), i32([[0, 1], [2, 3]]), i32([3, 9])
    ar.kv4_attention(Q, cache, t, n)
    for a in ((Q.float(), t, n), (Q[:, :3], t, n), (Q, t[:1], n), (Q, t, n[:1]), (Q, t.long(), n),
              (Q, t, n.float()), (Q[..., :32], t, n), (Q.transpose(0, 1), t, n), (Q[None, None], t, n),
              (torch.zeros((4, 2, 4, 64), dtype=torch.bfloat16, device=dev()).transpose(0, 1), t, n)):
        with pytest.raises(ValueError):
            ar.kv4_attention(a[0], cache, a[1], a[2])
    for kw in (dict(max_len=33), dict(max_len=-1), dict(scale=0.0), dict(scale=float("nan"))):
        with pytest.raises(ar.ArError):
            ar.kv4_attention(Q, cache, t, n, **kw)
    # nothing to do
    assert ar.kv4_attention(Q[:0], cache, t[:0], n[:0]).out.shape == (0, 4, 64)
    ar.kv4_write(K[:0], K[:0], cache, s[:0])
    assert ar.kv4_read(cache, s[:0])[0].shape == (0, 2, 64)
    none = ar.kv4_attention(Q, cache, t[:, :0].contiguous(), n, want_lse=True)
    assert (none.out == 0).all() and torch.isneginf(none.lse).all()


@pytest.mark.parametrize("lengths,new", [([1], 1), ([1, 70, 200], 1), ([3000, 90], 3)])
@pytest.mark.parametrize("size", [2.0 ** 13, 2.0 ** 17, 2.0 ** 40])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 32), (128, 128)])
def test_scores_beyond_2_to_28(lengths, new, size, D, group):
    """Scores so far apart that a row takes one key, or the mean of equal ones."""
    log(f"kv4 scores of {size}^2, {lengths} {new} x {D}")
    rng = np.random.default_rng(62)
    H, heads, P, B = 4, 1, 64, len(lengths)
    per = [-(-n // P) for n in lengths]
    cache = ar.kv4_cache(sum(per), heads, D, page_size=P, group_size=group)
    table, ks, vs = np.full((B, max(per)), -1), [], []
    for b, n in enumerate(lengths):
        at = sum(per[:b])
        table[b, :per[b]] = np.arange(at, at + per[b])
        level = size * rng.integers(1, 200, n)[:, None, None] * np.ones((1, heads, D))
        slots = i32(at * P + np.arange(n))
        ar.kv4_write(bf16(level)[0], bf16(rng.normal(size=(n, heads, D)))[0], cache, slots)
        k, v = ar.kv4_read(cache, slots, out_dtype=torch.float32)
        ks.append(k.double().cpu().numpy())
        vs.append(v.double().cpu().numpy())
    sign = np.where(np.arange(B * new * H) % 3 == 0, -1.0, 1.0).reshape(B, new, H, 1)
    Q, q = bf16(size * sign * np.ones(D))
    got = ar.kv4_attention(Q, cache, i32(table), i32(lengths), want_lse=True)
    out, lse = got.out.double().cpu().numpy(), got.lse.double().cpu().numpy()
    for b, n in enumerate(lengths):
        for h in range(H):
            o, l, w, _ = R.rows(q[b, :, h], ks[b][:, 0], vs[b][:, 0], R.causal(new, n), D ** -0.5)
            weight = np.stack([R.rows(q[b, i:i + 1, h], ks[b][:, 0], np.abs(vs[b][:, 0]).max(1)[:, None] / 7,
                                      R.causal(new, n)[i:i + 1], D ** -0.5)[0][0] for i in range(new)])
            bound = out_bound(o, w, 0.0 * l, D, n, W_BITS) + 2.0 ** -10 * weight
            check(out[b, :, h], o, bound, f"out {b} {h}")
            check(lse[b, :, h], l, np.abs(l) * (D + 8) * 2.0 ** -24 + 1e-3, f"lse {b} {h}")


def held_by(cache, n):
    """The first n tokens of a cache in float64."""
    return (x.double().cpu().numpy() for x in
            ar.kv4_read(cache, i32(np.arange(n)), out_dtype=torch.float32))


@pytest.mark.parametrize("D,group", [(64, 32), (128, 128)])
@pytest.mark.parametrize("n", [150, 3000])
@pytest.mark.parametrize("size", [2.0 ** 118, 1e37, 1.7e38])
def test_queries_at_the_top_of_their_range(size, n, D, group):
    """Keys of zeros leave scores of 0 whatever the queries; any other key is far from them."""
    log(f"kv4 queries of {size}, {n} x {D}")
    rng = np.random.default_rng(41)
    heads, H, P = 2, 8, 64
    pages = -(-n // P)
    q0 = size * np.clip(rng.normal(size=(1, 1, H, D)), -1, 1)
    Q, q = bf16(q0)
    for key in (None, 30, n - 1):
        cache = ar.kv4_cache(pages, heads, D, page_size=P, group_size=group)
        x = np.zeros((n, heads, D))
        if key is not None:     # along the first head's query: its score is the largest by far
            x[key] = 2e-29 * np.sign(q0[0, 0, 0])
        K, V = bf16(x)[0], bf16(rng.normal(size=(n, heads, D)))[0]
        ar.kv4_write(K, V, cache, i32(np.arange(n)))
        k, v = held_by(cache, n)
        for scale in (None, 0.5, 2.0 ** 20):
            got = ar.kv4_attention(Q, cache, i32(np.arange(pages)[None]), i32([n]), want_lse=True,
                                   scale=scale)
            out, lse = got.out.double().cpu().numpy()[0, 0], got.lse.cpu().numpy()[0, 0]
            for h in range(H):
                s = D ** -0.5 if scale is None else scale
                o, l, w, mag = R.rows(q[0, :, h], k[:, h // 4], v[:, h // 4], R.causal(1, n), s)
                # scores of 0 are exact; one that is not is beyond all others or below them by more
                # than its error (2^-17 of the largest product of a channel)
                far = s * (k[:, h // 4] @ q[0, 0, h])
                cut = D * 2.0 ** -17 * np.abs(q[0, 0, h]).max() * s * np.abs(k[:, h // 4]).max()
                assert key is None or abs(far[key]) > cut + 1000
                weight = np.abs(v[:, h // 4]).max() / 7
                bound = out_bound(o, w, np.zeros(1), D, n, W_BITS) + 2.0 ** -10 * weight
                check(out[h], o[0], bound[0], f"out {key} {h} {scale}")
                check(lse[h], l[0], lse_bound(l, mag, D, n)[0] + cut, f"lse {key} {h}")


@pytest.mark.parametrize("qs,ks_", [(2.0 ** -122, 2.0 ** 120), (2.0 ** -130, 2.0 ** 121),
                                    (2.0 ** -126, 2.0 ** 119)])
def test_queries_at_the_bottom_of_their_range(qs, ks_):
    """Tiny queries, subnormal ones among them, over huge keys."""
    log(f"kv4 queries of {qs}")
    rng = np.random.default_rng(42)
    H, heads, D, P, n = 8, 2, 64, 32, 150
    cache = ar.kv4_cache(8, heads, D, page_size=P, group_size=32)
    K, V = bf16(ks_ * rng.normal(size=(n, heads, D)))[0], bf16(rng.normal(size=(n, heads, D)))[0]
    ar.kv4_write(K, V, cache, i32(np.arange(n)))
    k, v = held_by(cache, n)
    Q, q = bf16(qs * rng.normal(size=(1, 1, H, D)))
    assert np.abs(q).max() > 0
    for scale in (None, 16.0):
        got = ar.kv4_attention(Q, cache, i32(np.arange(8)[None]), i32([n]), want_lse=True, scale=scale)
        compare(got, q, [k], [v], 1, f"tiny {qs}", scale=scale)


def compare_seen(got, q, ks, vs, new, what):
    """As compare, with bounds of what a row sees only: weights below 2^-30 of its own largest
    weight times scale may vanish."""
    B, _, H, D = q.shape
    out, lse = got.out.double().cpu().numpy().reshape(q.shape), got.lse.cpu().numpy().reshape(B, new, H)
    for b in range(B):
        n, r = len(ks[b]), H // ks[b].shape[1]
        sees = R.causal(new, n)
        for h in range(H):
            k, v = ks[b][:, h // r], vs[b][:, h // r]
            o, l, size, mag = R.rows(q[b, :, h], k, v, sees, D ** -0.5)
            cut = D * 2.0 ** -17 * np.abs(q[b, :, h]).max(1) * D ** -0.5 * np.abs(k).max() / 7
            weight = np.stack([R.rows(q[b, i:i + 1, h], k, np.abs(v).max(1)[:, None] / 7,
                                      sees[i:i + 1], D ** -0.5)[0][0] for i in range(new)])
            bound = out_bound(o, size, mag, D, n, W_BITS) + size * 2 * np.expm1(cut)[:, None] + \
                (2.0 ** -10 + n * 2.0 ** -27) * weight
            check(out[b, :, h], o, bound, f"{what}: out {b} {h}")
            check(lse[b, :, h], l, lse_bound(l, mag, D, n) + cut, f"{what}: lse {b} {h}")


VALUES = [  # lengths, new, heads, key heads, head_dim, page, group, further pages of the table
    ([90], 5, 4, 2, 64, 16, 32, 0), ([70, 33], 3, 8, 2, 128, 64, 128, 0),
    ([2500], 4, 8, 1, 128, 64, 64, 0), ([300], 3, 4, 1, 128, 32, 32, 0),
    ([700], 5, 14, 2, 64, 16, 32, 100), ([400, 90], 8, 8, 1, 128, 64, 128, 3100)]


@pytest.mark.parametrize("times", [20, 35, 70, 115])
@pytest.mark.parametrize("lengths,new,H,heads,D,P,group,more", VALUES)
def test_large_values_that_some_rows_do_not_see(lengths, new, H, heads, D, P, group, more, times):
    """The draft's last token has values 2^times times the others'; its earlier rows do not see it."""
    log(f"kv4 hidden values 2^{times} {lengths} {new} {H}/{heads} x {D} group {group}")
    rng = np.random.default_rng(times)
    cache, table, ks, vs = filled(rng, lengths, heads, D, P, group)
    for b, n in enumerate(lengths):
        slot = int(table[b, (n - 1) // P]) * P + (n - 1) % P
        K, V = bf16(keys(rng, 1, heads, D))[0], bf16(2.0 ** times * rng.normal(size=(1, heads, D)))[0]
        ar.kv4_write(K, V, cache, i32([slot]))
        for x, y in zip((ks, vs), ar.kv4_read(cache, i32([slot]), out_dtype=torch.float32)):
            x[b][n - 1] = y[0].double().cpu().numpy()
    if more:
        table = torch.cat([table, table[:, -1:].expand(-1, more)], 1).contiguous()
    Q, q = bf16(1.5 * rng.normal(size=(len(lengths), new, H, D)))
    got = ar.kv4_attention(Q, cache, table, i32(lengths), want_lse=True)
    compare_seen(got, q, ks, vs, new, "hidden")


@pytest.mark.parametrize("n", [1, 40, 70, 2500])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_large_values_that_weigh_little(n, group):
    """Tokens of values 2^60 whose weight is about 2^-100, in front of the others and behind
    them; and all values near 2^118, some of which no row can do without."""
    log(f"kv4 values that weigh little, {n} group {group}")
    rng = np.random.default_rng(n)
    heads, H, D, P = 1, 4, 128, 64
    pages = -(-n // P)
    q0 = np.zeros((1, 1, H, D))
    q0[..., 0] = 8.0                     # scores of a key: its first channel times 8/sqrt(128)
    Q, q = bf16(q0 + 0.01 * rng.normal(size=q0.shape))
    for where in ([], [0], [n - 1], [0, n // 2]):
        x, y = 0.1 * rng.normal(size=(n, heads, D)), rng.normal(size=(n, heads, D))
        x[:, :, 0] = 0.0
        x[where, :, 0] = -100.0          # e^-70, 2^-102
        y[where] *= 2.0 ** 60
        if not where:
            y *= 2.0 ** 118
            x[n // 3, :, 0] = 5.0
        cache = ar.kv4_cache(pages, heads, D, page_size=P, group_size=group)
        ar.kv4_write(bf16(x)[0], bf16(y)[0], cache, i32(np.arange(n)))
        k, v = held_by(cache, n)
        got = ar.kv4_attention(Q, cache, i32(np.arange(pages)[None]), i32([n]), want_lse=True)
        compare_seen(got, q, [k], [v], 1, f"little {where}")


@pytest.mark.parametrize("n,apart", [(900, 256), (3000, 128)])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 128)])
def test_values_near_the_top(n, apart, D, group):
    """Values of 2^119 whose weights rise from tile to tile: no sum comes near float32's end."""
    log(f"kv4 values of 2^119, {n} x {D}")
    heads, H, P = 2, 4, 64
    pages = -(-n // P)
    Q, q = bf16(np.broadcast_to(np.eye(1, D), (1, 1, H, D)))
    t = np.arange(n)
    x, y = np.zeros((n, heads, D)), np.full((n, heads, D), 2.0 ** 119)
    x[:, :, 0] = (t // apart % 2 * 7.5 - (t % 7 != 0) * 12.0)[:, None]
    y[..., 1::2] *= -1.5
    cache = ar.kv4_cache(pages, heads, D, page_size=P, group_size=group)
    ar.kv4_write(bf16(x)[0], bf16(y)[0], cache, i32(t))
    k, v = held_by(cache, n)
    scale = 0.6931471805599453
    got = ar.kv4_attention(Q, cache, i32(np.arange(pages)[None]), i32([n]), want_lse=True, scale=scale)
    compare(got, q, [k], [v], 1, "top", scale=scale)


KERNELS = [  # sequences, longest, tokens the table has room for, new, heads, key heads, head_dim, group
    (3, 900, 3000, 1, 8, 2, 64, 32),        # one tile of rows, divided
    (3, 900, 3000, 2, 8, 2, 64, 64),
    (3, 900, 3000, 1, 8, 2, 128, 32),
    (3, 900, 3000, 1, 8, 2, 128, 64),
    (3, 900, 3000, 1, 8, 2, 128, 128),
    (5, 200, 256, 1, 8, 2, 64, 32),         # undivided, four waves
    (5, 200, 256, 2, 8, 2, 64, 64),
    (5, 200, 256, 1, 8, 2, 128, 32),
    (5, 200, 256, 1, 8, 2, 128, 64),
    (5, 200, 256, 2, 8, 2, 128, 128),
    (3, 500, 1024, 3, 8, 2, 64, 32),        # undivided, eight waves
    (3, 500, 1024, 1, 8, 2, 64, 64),
    (3, 500, 1024, 1, 8, 2, 128, 32),
    (3, 500, 1024, 3, 8, 2, 128, 64),
    (3, 500, 1024, 1, 8, 2, 128, 128),
    (2, 900, 200000, 3, 12, 1, 64, 32),     # two tiles of rows, divided
    (2, 900, 200000, 3, 12, 1, 64, 64),
    (2, 900, 200000, 5, 12, 1, 128, 64),
    (2, 900, 200000, 3, 12, 1, 128, 128),
    (128, 300, 1024, 3, 24, 4, 64, 32),     # .. undivided
    (128, 300, 1024, 3, 24, 4, 64, 64),
    (128, 300, 1024, 5, 24, 4, 128, 64),
    (128, 300, 1024, 3, 24, 4, 128, 128),
    (160, 300, 2048, 3, 24, 4, 128, 128),   # of up to 2048 tokens
    (64, 900, 3000, 2, 16, 4, 64, 32),      # many rows to join
    (64, 900, 3000, 2, 16, 4, 128, 64),
    (512, 5000, 5008, 1, 4, 4, 64, 64),     # many sequences: one far longer than the others
    (512, 5000, 5008, 1, 4, 4, 128, 128),
]


@pytest.mark.parametrize("B,longest,room,new,H,heads,D,group", KERNELS)
def test_every_kernel(B, longest, room, new, H, heads, D, group):
    log(f"kv4 every kernel {B} x {longest} of {room} new {new} heads {H}/{heads} x {D} group {group}")
    rng = np.random.default_rng(B + new)
    P = 16
    lengths = [int(x) for x in rng.integers(0, 40, B)]
    lengths[B // 2] = longest
    cache, table, ks, vs = filled(rng, lengths, heads, D, P, group)
    wide = torch.full((B, room // P), -1, dtype=torch.int32, device=dev())
    n = min(table.shape[1], room // P)
    wide[:, :n] = table[:, :n]
    Q, q = bf16(1.5 * rng.normal(size=(B, new, H, D)))
    got = ar.kv4_attention(Q, cache, wide, i32(lengths), want_lse=True)
    compare(got, q, ks, vs, new, "every kernel")


@pytest.mark.parametrize("group", [32, 64, 128])
def test_scales_of_either_sign(group):
    """A cache that its owner filled: scales below 0, as large as they come."""
    log(f"kv4 negative scales, group {group}")
    rng = np.random.default_rng(71)
    heads, H, D, P, n = 2, 4, 128, 64, 300
    for size in (1.0, 1e30):
        codes = rng.integers(0, 256, (5, 2, heads, P, D // 2)).astype(np.uint8)
        scale = (rng.uniform(0.01, 0.1, (5, 2, heads, P, D // group)) *
                 rng.choice([-1.0, 1.0], (5, 2, heads, P, D // group))).astype(F32)
        scale[:, 1] *= F32(-size)
        scale[:, 1, 0] = -np.abs(scale[:, 1, 0])        # below 0 throughout
        k, v = R.held(codes, scale, np.arange(n))
        Q, q = bf16(rng.normal(size=(1, 1, H, D)))
        got = ar.kv4_attention(Q, on_gpu((codes, scale)), i32(np.arange(5)[None]), i32([n]), want_lse=True)
        compare(got, q, [k], [v], 1, f"signs {size}")
