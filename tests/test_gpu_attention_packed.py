"""attention_packed against the oracle in float64: lengths from one token to several tiles,
grouped heads, packed sequences, keys longer and shorter than queries, tokens that lie apart,
rows that see nothing, infinities where nobody looks, offsets that lead nowhere."""
import numpy as np
import pytest
import torch

from attention_common import bf16, check, i32, keys, lse_bound, oracle_heads, out_bound
from gpu_common import dev, log
from oracle import kv4_ref as R

pytestmark = pytest.mark.gpu
ar = pytest.importorskip("autoround_signsgd_rounding_amd")

P_BITS = 2.0 ** -8       # weights are rounded to bf16


def offsets(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(int)


def problem(seed, lq, lk, H, Hk, D):
    rng = np.random.default_rng(seed)
    q, k = 1.5 * rng.normal(size=(sum(lq), H, D)), keys(rng, sum(lk), Hk, D)
    v = rng.normal(size=(sum(lk), Hk, D))
    return bf16(q), bf16(k), bf16(v)


def verify(got, lse, q, k, v, qo, ko, scale, what):
    for b in range(len(qo) - 1):
        rows, cols = slice(qo[b], qo[b + 1]), slice(ko[b], ko[b + 1])
        nq, nk = qo[b + 1] - qo[b], ko[b + 1] - ko[b]
        if nq == 0:
            continue
        out, l, size, mag = oracle_heads(q[rows], k[cols], v[cols], R.causal(nq, nk), scale)
        D = q.shape[2]
        check(got[rows], out, out_bound(out, size, mag, D, nk, P_BITS), f"{what}: out {b}")
        if lse is not None:
            empty = np.isneginf(l)
            assert (np.isneginf(lse[rows]) == empty).all(), what
            check(lse[rows][~empty], l[~empty], lse_bound(l, mag, D, nk)[~empty], f"{what}: lse {b}")
            assert (got[rows][empty] == 0).all()


CASES = [  # queries, keys (None: the same), heads, key heads, head_dim
    ([1], None, 1, 1, 64),
    ([1, 1, 2], None, 4, 4, 128),
    ([37], None, 8, 8, 128),
    ([64, 63, 65], None, 4, 2, 64),
    ([130], None, 6, 2, 128),
    ([16, 1, 200, 3, 77], None, 8, 1, 128),
    ([129, 0, 31], None, 7, 1, 64),
    ([300], None, 2, 2, 128),
    ([700], None, 3, 1, 64),
    ([5, 17, 90], [5 + 200, 17 + 63, 90 + 64], 8, 2, 128),
    ([1], [513], 8, 2, 64),
    ([40, 3, 100], [10, 0, 99], 4, 2, 128),     # fewer keys than queries: rows that see nothing
    ([2, 2], [0, 0], 2, 1, 64),
    ([9], [70], 256, 1, 64),                    # the largest group
    ([3], [5], 300, 300, 64),                   # many key heads
]


@pytest.mark.parametrize("lq,lk,H,Hk,D", CASES)
def test_against_the_oracle(lq, lk, H, Hk, D):
    log(f"packed {lq} {lk} heads {H}/{Hk} x {D}")
    same, lk = lk is None, lq if lk is None else lk
    (Q, q), (K, k), (V, v) = problem(sum(lq) + H, lq, lk, H, Hk, D)
    qo, ko = offsets(lq), offsets(lk)
    r = ar.attention_packed(Q, K, V, i32(qo), k_offsets=None if same else i32(ko), want_lse=True)
    torch.cuda.synchronize()
    got, lse = r.out.double().cpu().numpy(), r.lse.cpu().numpy()
    verify(got, lse, q, k, v, qo, ko, D ** -0.5, "packed")
    again = ar.attention_packed(Q, K, V, i32(qo), k_offsets=None if same else i32(ko))
    assert again.lse is None and torch.equal(again.out, r.out)


def test_parts_of_one_product():
    """q, k and v side by side in one array, another scale, a given output."""
    log("packed strided")
    H, Hk, D, T = 4, 2, 64, 150
    rng = np.random.default_rng(5)
    qkv, x = bf16(rng.normal(size=(T, H + 2 * Hk, D)))
    Q, K, V = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device=dev())
    r = ar.attention_packed(Q, K, V, i32([3, 60, 140]), scale=0.25, out=out, want_lse=True)
    torch.cuda.synchronize()
    assert r.out is out
    got = out.double().cpu().numpy()
    assert (got[:3] == 7).all() and (got[140:] == 7).all()      # rows of no sequence
    q, k, v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    verify(got, r.lse.cpu().numpy(), q, k, v, [3, 60, 140], [3, 60, 140], 0.25, "parts")


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_hidden_infinities(bad):
    """A NaN or an infinity in a key or a value reaches the rows that see it, and no other:
    not those in front of it, not another sequence's."""
    log(f"packed hidden {bad}")
    lq, H, Hk, D = [70, 130, 64], 4, 2, 128
    rng = np.random.default_rng(9)
    (Q, q), (K, k), (V, v) = problem(8, lq, lq, H, Hk, D)
    qo = offsets(lq)
    want = ar.attention_packed(Q, K, V, i32(qo)).out
    for t, which in ((qo[1] + 100, "v"), (qo[1] + 3, "k"), (qo[0] + 69, "v"), (qo[2], "k")):
        X = {"k": K.clone(), "v": V.clone()}
        X[which][t, 1, 5] = bad
        r = ar.attention_packed(Q, X["k"], X["v"], i32(qo), want_lse=True)
        torch.cuda.synchronize()
        b = int(np.searchsorted(qo, t, side="right")) - 1
        clean = np.ones((sum(lq), H), bool)
        clean[t:qo[b + 1], H // Hk:] = False
        clean = torch.from_numpy(clean).to(dev())
        d = (r.out.double() - want.double())[clean].abs()
        # the rows that are done again round their weights less: both are within the bound
        assert d.max().item() <= 0.05, (t, which)
        assert torch.isfinite(r.out[clean]).all()
        hit = r.out[t:qo[b + 1], H // Hk:]
        if which == "v":
            assert not torch.isfinite(hit[..., 5]).any()
            assert torch.isfinite(hit[..., 6]).all()
            if np.isinf(bad):
                assert (hit[..., 5] == bad).all()
        elif np.isnan(bad):
            assert torch.isnan(hit).all() and torch.isnan(r.lse[t:qo[b + 1], H // Hk:]).all()
    # exact values of rows done again
    V2 = V.clone()
    V2[qo[1] + 129, 0, 0] = bad
    got = ar.attention_packed(Q, K, V2, i32(qo)).out.double().cpu().numpy()
    sl = slice(qo[1], qo[1] + 129)
    out, _, size, mag = oracle_heads(q[sl], k[sl], v[sl], R.causal(129, 129), D ** -0.5)
    check(got[sl], out, out_bound(out, size, mag, D, 129, P_BITS), "rows done again")


def test_extreme_scores():
    """Rows whose weight is all on one key, scores in the thousands, equal scores."""
    log("packed extreme scores")
    H, D, T = 2, 64, 200
    rng = np.random.default_rng(1)
    (Q, q), (K, k), (V, v) = problem(2, [T], [T], H, H, D)
    Q[50:100] *= 64
    K[::7] *= 16
    Q[100:120] = 0
    q, k = Q.double().cpu().numpy(), K.double().cpu().numpy()
    r = ar.attention_packed(Q, K, V, i32([0, T]), want_lse=True)
    torch.cuda.synchronize()
    verify(r.out.double().cpu().numpy(), r.lse.cpu().numpy(), q, k, v, [0, T], [0, T], D ** -0.5,
           "extreme")


def test_large_values():
    log("packed large values")
    (Q, q), (K, k), (V, v) = problem(4, [90], [90], 2, 2, 64)
    V = V * 1e30
    v = V.double().cpu().numpy()
    got = ar.attention_packed(Q, K, V, i32([0, 90])).out.double().cpu().numpy()
    verify(got, None, q, k, v, [0, 90], [0, 90], 0.125, "large values")


@pytest.mark.parametrize("qo", [[0, 500, 100], [-5, 60, 1 << 30], [90, 20, 50, 10], [200, 300, 400],
                                [-1 << 31, (1 << 31) - 1], [0, 0, 0]])
def test_offsets_that_lead_nowhere(qo):
    """Offsets outside the arrays are clamped, decreasing ones give something; nothing
    outside the output is written."""
    log(f"packed offsets {qo}")
    T, H, D = 96, 4, 64
    (Q, _), (K, _), (V, _) = problem(3, [T], [T], H, 2, D)
    whole = torch.full((T + 64, H, D), 7.0, dtype=torch.bfloat16, device=dev())
    ar.attention_packed(Q, K, V, i32(qo), out=whole[32:32 + T])
    ar.attention_packed(Q, K, V, i32(qo), k_offsets=i32(qo[::-1]), out=whole[32:32 + T])
    torch.cuda.synchronize()
    assert (whole[:32] == 7).all() and (whole[32 + T:] == 7).all()


@pytest.mark.parametrize("qo", [[0, 9000, 100], [-5, 60, 1 << 30], [9000, 20, 5000, 10], [0, 6000, 0, 6000],
                                [-1 << 31, (1 << 31) - 1], [6000, 6000]])
def test_offsets_that_lead_nowhere_in_divided_calls(qo):
    """The same where the keys are divided, sequences over each other among them."""
    log(f"packed divided offsets {qo}")
    T, H, D = 6000, 4, 64
    (Q, _), (K, _), (V, _) = problem(3, [T], [T], H, 2, D)
    whole = torch.full((T + 64, H, D), 7.0, dtype=torch.bfloat16, device=dev())
    ar.attention_packed(Q, K, V, i32(qo), out=whole[32:32 + T])
    ar.attention_packed(Q, K, V, i32(qo), k_offsets=i32(qo[::-1]), out=whole[32:32 + T])
    torch.cuda.synchronize()
    assert (whole[:32] == 7).all() and (whole[32 + T:] == 7).all()


def test_many_sequences():
    """More sequences than a wave has lanes, most of them short or empty."""
    log("packed many sequences")
    rng = np.random.default_rng(11)
    lq = [int(x) for x in rng.choice([0, 1, 2, 5, 40], size=300)]
    (Q, q), (K, k), (V, v) = problem(12, lq, lq, 2, 1, 64)
    qo = offsets(lq)
    got = ar.attention_packed(Q, K, V, i32(qo)).out.double().cpu().numpy()
    verify(got, None, q, k, v, qo, qo, 0.125, "many")


@pytest.mark.parametrize("T,H,Hk,D", [(4096, 8, 1, 128), (9000, 2, 2, 64)])
def test_long_against_float64(T, H, Hk, D):
    """Long prompts, against float64 on the GPU row by row of heads."""
    log(f"packed long {T} {H}/{Hk} x {D}")
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    q, k, v = (torch.randn((T, h, D), generator=g, device="cuda").to(torch.bfloat16)
               for h in (H, Hk, Hk))
    r = ar.attention_packed(q, k, v, i32([0, T]), want_lse=True)
    for h in range(H):
        x = (q[:, h].double() @ k[:, h // (H // Hk)].double().t()) * D ** -0.5
        x = x.masked_fill(torch.ones((T, T), dtype=torch.bool, device="cuda").triu(1), -np.inf)
        lse = torch.logsumexp(x, 1)
        p = torch.exp(x - lse[:, None])
        vh = v[:, h // (H // Hk)].double()
        out, size = p @ vh, p @ vh.abs()
        mag = D ** -0.5 * (q[:, h].double().abs() @ k[:, h // (H // Hk)].double().abs().t()).amax(1)
        b = out_bound(out.cpu().numpy(), size.cpu().numpy(), mag.cpu().numpy(), D, T, P_BITS)
        check(r.out[:, h].double().cpu().numpy(), out.cpu().numpy(), b, "long")
        check(r.lse[:, h].double().cpu().numpy(), lse.cpu().numpy(),
              lse_bound(lse.cpu().numpy(), mag.cpu().numpy(), D, T), "long lse")


def test_few_queries_behind_a_long_prefix():
    """A chunk of a few tokens behind thousands: the keys' axis is what there is to divide."""
    log("packed chunk")
    lq, lk = [3, 20], [5000, 2777]
    (Q, q), (K, k), (V, v) = problem(21, lq, lk, 8, 2, 128)
    qo, ko = offsets(lq), offsets(lk)
    r = ar.attention_packed(Q, K, V, i32(qo), k_offsets=i32(ko), want_lse=True)
    verify(r.out.double().cpu().numpy(), r.lse.cpu().numpy(), q, k, v, qo, ko, 128 ** -0.5, "chunk")


def test_many_sequences_of_which_few_are_long():
    """More sequences than a wave has lanes, the keys of two divided."""
    log("packed few long ones of many")
    rng = np.random.default_rng(13)
    lq = [int(x) for x in rng.integers(0, 3, 100)]
    lk = [int(x) for x in rng.integers(0, 60, 100)]
    lq[5], lk[5], lq[80], lk[80] = 2, 3100, 1, 2600
    (Q, q), (K, k), (V, v) = problem(14, lq, lk, 4, 1, 128)
    qo, ko = offsets(lq), offsets(lk)
    r = ar.attention_packed(Q, K, V, i32(qo), k_offsets=i32(ko), want_lse=True)
    verify(r.out.double().cpu().numpy(), r.lse.cpu().numpy(), q, k, v, qo, ko, 128 ** -0.5, "few")


def test_divided_keys_and_hidden_infinities():
    """The last part of the keys holds an infinity that only the later queries see."""
    log("packed divided, hidden infinity")
    lq, lk, H, Hk, D = [40], [5000], 4, 2, 64
    (Q, q), (K, k), (V, v) = problem(22, lq, lk, H, Hk, D)
    V[4990, 0, 5] = np.inf
    r = ar.attention_packed(Q, K, V, i32([0, 40]), k_offsets=i32([0, 5000]), want_lse=True)
    got, lse = r.out.double().cpu().numpy(), r.lse.cpu().numpy()
    out, l, size, mag = oracle_heads(q, k, v, R.causal(40, 5000), D ** -0.5)
    bound = out_bound(out, size, mag, D, 5000, P_BITS)
    check(got[:30], out[:30], bound[:30], "in front of it")
    check(got[30:, 2:], out[30:, 2:], bound[30:, 2:], "the other key head's")
    check(lse, l, lse_bound(l, mag, D, 5000), "lse")
    assert (got[30:, :2, 5] == np.inf).all()


@pytest.mark.parametrize("bad", [None, np.nan])
def test_many_tiles(bad):
    """More workgroups than run at once: prompts of very different lengths, 64 heads; rows in
    front of a NaN among the values."""
    log(f"packed many tiles {bad}")
    lq, H, Hk, D = [1000, 1, 0, 700, 31, 32, 33, 1200, 64, 200], 64, 8, 128
    (Q, q), (K, k), (V, v) = problem(23, lq, lq, H, Hk, D)
    qo = offsets(lq)
    if bad is not None:
        V[qo[1] - 1, 1] = bad                  # the last token of the first sequence
    r = ar.attention_packed(Q, K, V, i32(qo), want_lse=True)
    got, lse = r.out.double().cpu().numpy(), r.lse.cpu().numpy()
    hit = got[qo[1] - 1, 8:16].copy()
    assert np.isnan(hit).all() == (bad is not None)
    for h in (0, 13, 63):
        if bad is not None and h // 8 == 1:
            got[qo[1] - 1, h] = 0
            o = oracle_heads(q[:1000, h:h + 1], k[:1000, 1:2], v[:1000, 1:2], R.causal(1000, 1000),
                             D ** -0.5)
            check(got[:999, h:h + 1], o[0][:999],
                  out_bound(o[0], o[2], o[3], D, 1000, P_BITS)[:999], "in front of it")
            continue
        one = lambda x, i: x[:, i:i + 1]        # noqa: E731
        verify(one(got, h), one(lse, h), one(q, h), one(k, h // 8), one(v, h // 8), qo, qo,
               D ** -0.5, f"many tiles {h}")


def test_tokens_far_apart():
    """Tokens at the largest stride: offsets pass 2^32 elements."""
    log("packed far apart")
    H, Hk, D, T, S = 4, 2, 128, 1100, (1 << 22) - 8
    rng = np.random.default_rng(24)
    base = torch.empty(T * S, dtype=torch.bfloat16, device=dev())
    x = base.view(T, S)[:, :(H + 2 * Hk) * D].unflatten(1, (H + 2 * Hk, D))
    X, f = bf16(rng.normal(size=x.shape))
    x.copy_(X)
    qo = offsets([1060, 40])
    r = ar.attention_packed(x[:, :H], x[:, H:H + Hk], x[:, H + Hk:], i32(qo), want_lse=True)
    verify(r.out.double().cpu().numpy(), r.lse.cpu().numpy(), f[:, :H], f[:, H:H + Hk],
           f[:, H + Hk:], qo, qo, D ** -0.5, "far apart")
    del base, x
    torch.cuda.empty_cache()


def test_equals_the_blocks_attention():
    """Sequences of one length and a key head for each query head: ar_attention's case."""
    log("packed beside ar_attention")
    H, D, S, B = 4, 128, 200, 3
    (Q, _), (K, _), (V, _) = problem(6, [S] * B, [S] * B, H, H, D)
    dims = ar.block_dims(H * D, H, 64, S, B)
    flat = [x.reshape(S * B, H * D).contiguous() for x in (Q, K, V)]
    want = ar.attention(*flat, dims).view(S * B, H, D).double()
    got = ar.attention_packed(Q, K, V, i32(offsets([S] * B))).out.double()
    # both within their roundings of the same values (|v| below 5)
    assert (got - want).abs().max().item() <= 2.0 ** -8 * 2 * 5
    assert ((got - want).norm() / want.norm()).item() <= 2.0 ** -8


def test_binding_checks():
    (Q, _), (K, _), (V, _) = problem(6, [8], [8], 4, 2, 64)
    o = i32([0, 8])
    ar.attention_packed(Q, K, V, o)
    bad = [(Q.float(), K, V, o), (Q, K.half(), V, o), (Q[0], K, V, o), (Q, K, V[:4], o),
           (Q[:, :3], K, V, o), (Q, K, V, o.long()), (Q, K, V, o.cpu()), (Q.cpu(), K, V, o),
           (Q, K, V, o[None]), (Q[:4], K, V, o), (Q.transpose(0, 1), K, V, o),
           (Q, K[..., ::2].repeat(1, 1, 2)[..., ::2], V, o), (Q, K, V, i32([]))]
    for a in bad:
        with pytest.raises(ValueError):
            ar.attention_packed(*a)
    odd = torch.zeros((8, 4 * 64 + 4), dtype=torch.bfloat16, device=dev())[:, :256].view(8, 4, 64)
    for kw in (dict(out=torch.empty_like(Q)[:4]), dict(out=Q.float()), dict(k_offsets=i32([0])),
               dict(stream=torch.cuda.Stream(device=0), out=Q.cpu())):
        with pytest.raises(ValueError):
            ar.attention_packed(Q, K, V, o, **kw)
    with pytest.raises(ValueError):
        ar.attention_packed(odd, K, V, o)
    for s in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ar.ArError):
            ar.attention_packed(Q, K, V, o, scale=s)
    e = ar.attention_packed(Q[:0], K[:0], V[:0], i32([0, 0]), want_lse=True)
    assert e.out.shape == (0, 4, 64) and e.lse.shape == (0, 4)
    assert ar.attention_packed(Q, K, V, i32([0])).out.shape == Q.shape


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("lq,lk", [([40, 3, 200], [10, 2, 70]),
                                   ([40, 10, 300], [12, 4000, 290])])     # (keys divided)
def test_rows_without_a_key_beside_infinities(lq, lk, bad, D):
    """Fewer keys than queries: the first rows see no key and are 0, whatever the values hold that
    the rows behind them see; those are as without it, but for the channel concerned."""
    log(f"packed rows without a key beside {bad}, {lq} {lk} x {D}")
    H, Hk = 4, 2
    (Q, q), (K, k), (V, v) = problem(31, lq, lk, H, Hk, D)
    qo, ko = offsets(lq), offsets(lk)
    for at in (0, 5, -1):                # seen by every row with a key, by some, by the last
        for b in (0, 2):
            X, t = V.clone(), at % lk[b]
            X[ko[b] + t, 1, 9] = bad
            r = ar.attention_packed(Q, K, X, i32(qo), k_offsets=i32(ko), want_lse=True)
            got, lse = r.out.double().cpu().numpy(), r.lse.cpu().numpy()
            none = np.zeros((sum(lq), H), bool)
            for s in range(3):
                none[qo[s]:qo[s] + max(0, lq[s] - lk[s])] = True
            assert none.any() and (got[none] == 0).all() and np.isneginf(lse[none]).all()
            first = qo[b] + lq[b] - lk[b] + t            # the first row that sees it
            hit = got[first:qo[b + 1], H // Hk:, 9]
            assert (np.isnan(hit) if np.isnan(bad) else hit == bad).all()
            hit[:] = 0.0
            for s in range(3):
                rows, cols = slice(qo[s], qo[s + 1]), slice(ko[s], ko[s + 1])
                o, l, size, mag = oracle_heads(q[rows], k[cols], v[cols], R.causal(lq[s], lk[s]),
                                               D ** -0.5)
                if s == b:
                    o[first - qo[b]:, H // Hk:, 9] = 0.0
                check(got[rows], o, out_bound(o, size, mag, D, lk[s], P_BITS), f"out {s}")
                some = ~none[rows]
                check(lse[rows][some], l[some], lse_bound(l, mag, D, lk[s])[some], f"lse {s}")


@pytest.mark.parametrize("T", [200, 1000, 3000])
@pytest.mark.parametrize("D", [64, 128])
def test_values_near_the_top(T, D):
    """Values of 2^120 whose weights rise from tile to tile: no sum comes near float32's end."""
    log(f"packed values of 2^120, {T} x {D}")
    H, Hk = 4, 2
    (Q, _), (K, _), (V, _) = problem(51, [T], [T], H, Hk, D)
    # one channel of the keys holds the score, in halves of a power of two of the weight
    Q.zero_()
    K.zero_()
    Q[..., 0] = 1.0
    t = torch.arange(T, device=dev())
    K[..., 0] = ((t // 64 % 16) * 0.5 - (t % 7 != 0) * 12.0)[:, None].to(torch.bfloat16)
    V.fill_(2.0 ** 120)
    V[..., 1::2] *= -1.5
    q, k, v = (x.double().cpu().numpy() for x in (Q, K, V))
    scale = 0.6931471805599453
    r = ar.attention_packed(Q, K, V, i32([0, T]), want_lse=True, scale=scale)
    verify(r.out.double().cpu().numpy(), r.lse.cpu().numpy(), q, k, v, [0, T], [0, T], scale, "top")


@pytest.mark.parametrize("lq,lk", [([1], [1]), ([3, 70, 200], [3, 70, 200]), ([20, 9], [3000, 90])])
@pytest.mark.parametrize("size", [2.0 ** 13, 2.0 ** 17, 2.0 ** 40])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_beyond_2_to_28(lq, lk, size, D):
    """Scores so far apart that a row takes one key, or the mean of equal ones."""
    log(f"packed scores of {size}^2, {lq} {lk} x {D}")
    H, Hk = 4, 2
    (Q, q), (K, k), (V, v) = problem(61, lq, lk, H, Hk, D)
    qo, ko = offsets(lq), offsets(lk)
    # q is size or -size throughout, or as it was; keys are size times a whole number
    sign = torch.where(torch.arange(sum(lq), device=dev()) % 3 == 0, -1.0, 1.0)
    Q[:, :3] = (size * sign)[:, None, None].to(torch.bfloat16)
    level = torch.from_numpy(np.random.default_rng(7).integers(1, 200, sum(lk))).to(dev())
    K[:] = (size * level)[:, None, None].to(torch.bfloat16)
    q, k = Q.double().cpu().numpy(), K.double().cpu().numpy()
    r = ar.attention_packed(Q, K, V, i32(qo), k_offsets=i32(ko), want_lse=True)
    got, lse = r.out.double().cpu().numpy(), r.lse.double().cpu().numpy()
    for b in range(len(lq)):
        rows, cols = slice(qo[b], qo[b + 1]), slice(ko[b], ko[b + 1])
        # (scores of a row and a level are equal to the last bit: their sums go the same way)
        o, l, size_, _ = oracle_heads(q[rows, :3], k[cols][:, [0, 0, 1]], v[cols][:, [0, 0, 1]],
                                      R.causal(lq[b], lk[b]), D ** -0.5)
        check(got[rows, :3], o, out_bound(o, size_, 0.0 * l, D, lk[b], P_BITS), f"out {b}")
        check(lse[rows, :3], l, np.abs(l) * (D + 8) * 2.0 ** -24 + 1e-3, f"lse {b}")


F32_CASES = [  # queries, keys, heads, key heads, head_dim
    ([1], [1], 2, 1, 64), ([130, 1, 37], [130, 1, 37], 6, 2, 128), ([700], [700], 3, 1, 64),
    ([40, 3, 100], [10, 0, 99], 4, 2, 128), ([3, 20], [5000, 2777], 8, 2, 128),     # (keys divided)
    ([5, 17], [4000, 90], 4, 2, 64), ([600, 33, 500], [600, 33, 500], 64, 32, 128)]


@pytest.mark.parametrize("lq,lk,H,Hk,D", F32_CASES)
def test_float32_weights(lq, lk, H, Hk, D):
    """Weights in three bf16 parts: 2^-24 of each, and three sums for each key."""
    log(f"packed float32 weights {lq} {lk} heads {H}/{Hk} x {D}")
    (Q, q), (K, k), (V, v) = problem(sum(lq) + H, lq, lk, H, Hk, D)
    qo, ko = offsets(lq), offsets(lk)
    r = ar.attention_packed(Q, K, V, i32(qo), k_offsets=i32(ko), want_lse=True, float32_weights=True)
    got, lse = r.out.double().cpu().numpy(), r.lse.cpu().numpy()
    plain = ar.attention_packed(Q, K, V, i32(qo), k_offsets=i32(ko), want_lse=True)
    assert torch.equal(plain.lse, r.lse)
    worse = plain.out.double().cpu().numpy()
    for b in range(len(lq)):
        rows, cols = slice(qo[b], qo[b + 1]), slice(ko[b], ko[b + 1])
        o, l, size, mag = oracle_heads(q[rows], k[cols], v[cols], R.causal(lq[b], lk[b]), D ** -0.5)
        check(got[rows], o, out_bound(o, size, mag, D, 2 * lk[b], 2.0 ** -24), f"f32 weights: out {b}")
        assert (got[rows][np.isneginf(l)] == 0).all() and (np.isneginf(lse[rows]) == np.isneginf(l)).all()
        if lk[b] >= 500:        # what rounding the output alone costs
            error = lambda x: np.linalg.norm(x[rows] - o) / np.linalg.norm(o)       # noqa: E731
            assert error(got) <= 2.0 ** -9 and error(got) < error(worse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = ar.attention_packed(Q, K, V, i32(qo), k_offsets=i32(ko), float32_weights=True, stream=s)
    s.synchronize()
    assert torch.equal(again.out, r.out)


@pytest.mark.parametrize("bad", [np.nan, -np.inf])
def test_float32_weights_and_hidden_infinities(bad):
    """Values that a row does not see, with float32 weights as without; and scores far apart."""
    log(f"packed float32 weights, hidden {bad}")
    lq, H, Hk, D = [70, 130], 4, 2, 128
    (Q, q), (K, k), (V, v) = problem(8, lq, lq, H, Hk, D)
    V[199, 0, 0] = bad
    Q[30:60] *= 2.0 ** 20
    q = Q.double().cpu().numpy()
    r = ar.attention_packed(Q, K, V, i32([0, 70, 200]), want_lse=True, float32_weights=True)
    got = r.out.double().cpu().numpy()
    for rows, n in ((slice(0, 30), 70), (slice(70, 199), 130)):
        cols = slice(rows.start, rows.start + n)
        o, _, size, mag = oracle_heads(q[cols], k[cols], v[cols], R.causal(n, n), D ** -0.5)
        m = rows.stop - rows.start
        check(got[rows], o[:m], out_bound(o, size, mag, D, 2 * n, 2.0 ** -24)[:m], f"{rows}")
    assert torch.isfinite(r.out[30:60]).all() and torch.isfinite(r.lse).all()
    assert not torch.isfinite(r.out[199, 0, 0]) and torch.isfinite(r.out[199, 0, 1:]).all()


def test_float32_weights_equal_the_blocks_attention():
    """ar_attention's case: the same float32 values but for their sums' order, rounded to bf16."""
    log("packed float32 weights beside ar_attention")
    H, D, S, B = 4, 128, 200, 3
    (Q, _), (K, _), (V, _) = problem(6, [S] * B, [S] * B, H, H, D)
    dims = ar.block_dims(H * D, H, 64, S, B)
    flat = [x.reshape(S * B, H * D).contiguous() for x in (Q, K, V)]
    want = ar.attention(*flat, dims).view(S * B, H, D).double()
    got = ar.attention_packed(Q, K, V, i32(offsets([S] * B)), float32_weights=True).out.double()
    # one step of bf16 apart at most, beside 1e-4 of the largest value for scores and sums
    assert ((got - want).abs() <= 2.0 ** -7 * want.abs() + 1e-4 * V.double().abs().max()).all()
    assert ((got - want).norm() / want.norm()).item() <= 2.0 ** -12
