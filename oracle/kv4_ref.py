"""Attention and the 4-bit key/value cache, from their definitions in
include/autoround_hip.h: codes and scales in float32 steps, everything else in float64."""
import numpy as np

F32 = np.float32


def grid(x, group):
    """Codes uint8 [.., D] and scales float32 [.., D/group] of x [.., D]."""
    x = np.asarray(x, F32)
    g = x.reshape(*x.shape[:-1], -1, group)
    with np.errstate(all="ignore"):
        lo = np.minimum(g.min(-1), F32(0))
        hi = np.maximum(g.max(-1), F32(0))
        d = hi - lo
        s = np.maximum(d / F32(15), F32(2.0 ** -100))
        zp = np.clip(np.rint(-lo / s), 0, 15)
        ok = np.isfinite(d)
        bits = (s.astype(F32).view(np.uint32) & ~np.uint32(15)) | np.where(ok, zp, 0).astype(np.uint32)
        s = np.where(ok, bits, np.uint32(0x7FC00000)).astype(np.uint32).view(F32)
        code = np.clip(np.rint(g / s[..., None]) + zp[..., None], 0, 15)
        code = np.where(ok[..., None], code, 0).astype(np.uint8)
    return code.reshape(x.shape), s


def value_byte(t, byte, half):
    """Where byte 32b + 16c + n of token t lies among a page's and head's value bytes."""
    b, c, n = byte // 32, byte // 16 % 2, byte % 16
    return (((t // 8 * (half // 32) + b) * 16 + n) * 8 + t % 8) * 2 + c


def write(codes, scale, k, v, slots):
    """Tokens k, v [T, heads, D] into the arrays of a cache, in place."""
    pages, _, heads, P, half = codes.shape
    for which, x in enumerate((k, v)):
        code, s = grid(x, 2 * half // scale.shape[4])
        packed = code[..., 0::2] | (code[..., 1::2] << 4)
        for i, slot in enumerate(slots):
            if not 0 <= slot < pages * P:
                continue
            p, t = slot // P, slot % P
            scale[p, which, :, t] = s[i]
            if which == 0:
                codes[p, 0, :, t] = packed[i]
            else:
                at = value_byte(t, np.arange(half), half)
                codes[p, 1].reshape(heads, P * half)[:, at] = packed[i]


def held(codes, scale, slots):
    """float64 keys and values [T, heads, D] of the slots, zeros for one outside the cache."""
    pages, _, heads, P, half = codes.shape
    G = scale.shape[4]
    out = np.zeros((2, len(slots), heads, 2 * half))
    for i, slot in enumerate(slots):
        if not 0 <= slot < pages * P:
            continue
        p, t = slot // P, slot % P
        at = value_byte(t, np.arange(half), half)
        for which in (0, 1):
            raw = codes[p, 0, :, t] if which == 0 else codes[p, 1].reshape(heads, P * half)[:, at]
            c = np.stack((raw & 15, raw >> 4), -1).reshape(heads, G, -1).astype(np.float64)
            s = scale[p, which, :, t]
            zp = (np.ascontiguousarray(s).view(np.uint32) & 15).astype(np.float64)
            out[which, i] = ((c - zp[..., None]) * s.astype(np.float64)[..., None]).reshape(heads, -1)
    return out[0], out[1]


def rows(q, k, v, sees, scale):
    """Rows q [n, D] over keys k [m, D] and values v, row i seeing those of sees [n, m]
    (bool). Returns out, lse, and what bounds of errors are made of: sum p|v| [n, D] and the
    largest scale·sum|q·k| of a key seen [n]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    out = np.zeros((len(q), v.shape[1]))
    lse, size, mag = np.full(len(q), -np.inf), np.zeros_like(out), np.zeros(len(q))
    for i in range(len(q)):
        at = np.flatnonzero(sees[i])
        if len(at) == 0:
            continue
        x = scale * (k[at] @ q[i])
        top = x.max()
        p = np.exp(x - top)
        lse[i] = top + np.log(p.sum())
        p /= p.sum()
        out[i], size[i] = p @ v[at], p @ np.abs(v[at])
        mag[i] = scale * (np.abs(k[at]) @ np.abs(q[i])).max()
    return out, lse, size, mag


def causal(nq, nk):
    """[nq, nk]: query i sees the keys 0 .. i + nk - nq."""
    return np.arange(nk)[None] <= np.arange(nq)[:, None] + (nk - nq)
