"""Plain 64-bit implementations of the 4-bit paged cache's operators, from the
formulas in include/fa.h: the format, the quantising append, reading back, and
attention over the cache."""
import numpy as np


def words(scale, zero):
    """int32 words of scales (that are bf16 values) and zeros (that are fp16 values)."""
    s = np.asarray(scale, np.float32).view(np.uint32)
    assert not np.any(s & 0xFFFF)
    z = np.asarray(zero, np.float16).view(np.uint16).astype(np.uint32)
    return (s | z).view(np.int32)


def unpack_words(w):
    """(scale, zero) in float64."""
    u = np.ascontiguousarray(w).view(np.uint32)
    return ((u & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64),
            (u & np.uint32(0xFFFF)).astype(np.uint16).view(np.float16).astype(np.float64))


def pack(c):
    """Codes [..., d] to bytes [..., d / 2]."""
    c = c.astype(np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def values(codes, w):
    """Rows of values [..., d] in float64."""
    s, z = unpack_words(w)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1).astype(np.float64)
    group = c.shape[-1] // w.shape[-1]
    return (c - np.repeat(z, group, -1)) * np.repeat(s, group, -1)


def bf16_at_least(t):
    """The smallest bf16 that is not below t >= 0 (fp32)."""
    t = np.float32(t)
    bits = int(t.view(np.uint32))
    up = (bits + 0xFFFF) // 0x10000 * 0x10000
    return np.uint32(up).view(np.float32)


def quantise(row, group):
    """One row [d] of float64 (16-bit values): (codes [d], scale, zero [d / group])."""
    codes, scale, zero = [], [], []
    for g in range(0, len(row), group):
        x = row[g:g + group]
        if not np.all(np.isfinite(x)):
            codes += [0] * group
            scale.append(np.float32(np.nan))
            zero.append(0.0)
            continue
        lo, hi = x.min(), x.max()
        # in sixteenths, so that fp32 holds the difference of any two
        wide = np.float32(np.float32((hi - lo) / 16) / np.float32(0.9375))
        s = bf16_at_least(max(wide, np.float32(np.abs(x).max() / 2048)))
        n = np.rint(x / np.float64(s)) if s > 0 else np.zeros(group)
        codes += list(np.minimum(n - n.min(), 15))
        scale.append(s)
        zero.append(-n.min() + 0.0)
    return np.array(codes), np.array(scale, np.float32), np.array(zero)


def append(x, slots, codes, w, bs, group):
    """x [T, Hkv, d] float64; returns new codes and words."""
    codes, w = codes.copy(), w.copy()
    blocks = codes.shape[0]
    for t, slot in enumerate(slots):
        if 0 <= slot < blocks * bs:
            for h in range(x.shape[1]):
                c, s, z = quantise(x[t, h], group)
                codes[slot // bs, h, slot % bs] = pack(c)
                nan = np.isnan(s)
                w[slot // bs, h, slot % bs] = np.where(nan, np.int32(0x7FC00000), words(np.where(nan, 0, s), z))
    return codes, w


def gathered(codes, w, table_row, n, bs):
    """The first n tokens of a request, [Hkv, n, d] float64; entries outside the pool read zeros."""
    blocks, Hkv, _, half = codes.shape
    out = np.zeros((Hkv, n, 2 * half))
    for i in range(-(-n // bs)):
        block = int(table_row[i])
        k = min(bs, n - i * bs)
        if 0 <= block < blocks:
            out[:, i * bs:i * bs + k] = values(codes[block, :, :k], w[block, :, :k])
    return out


def decode(q, kc, vc, kw, vw, table, lens, max_len, scale, mask, bs):
    """(o, lse, spread, reach, big) in float64: spread [B, H, Sq, d] is sum p s (|c - z|) (what rounding a
    weight is relative to), reach the largest of a row's sums of |q| times 15 scales and the zeros' share
    (what fp32 sums of scores are relative to), big [B, H, Sq, d] sum p s (15 + |z|) (what sums of O are)."""
    B, H, Sq, d = q.shape
    Hkv = kc.shape[1]
    o, spread, big = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q)
    lse, reach = np.full((B, H, Sq), -np.inf), np.zeros((B, H, Sq))
    group = d // kw.shape[-1]
    for b in range(B):
        L = min(max(int(lens[b]), 0), max_len)
        if L == 0:
            continue
        k, v = gathered(kc, kw, table[b], L, bs), gathered(vc, vw, table[b], L, bs)
        size = []  # s (15 + |z|) of every component's group
        for w in (kw, vw):
            x = np.zeros((Hkv, L, d))
            for i in range(-(-L // bs)):
                block, n = int(table[b, i]), min(bs, L - i * bs)
                if 0 <= block < len(w):
                    s, z = unpack_words(w[block, :, :n])
                    x[:, i * bs:i * bs + n] = np.repeat(s * (15 + np.abs(z)), group, -1)
            size.append(x)
        for h in range(H):
            g = h // (H // Hkv)
            x = q[b, h] @ k[g].T * scale
            for i in range(Sq):
                n = L if mask == "none" else min(L, max(0, L - Sq + i + 1))
                if n == 0:
                    continue
                xi = x[i, :n]
                top = xi.max()
                p = np.exp(xi - top)
                lse[b, h, i] = top + np.log(p.sum())
                p = p / p.sum()
                o[b, h, i] = p @ v[g, :n]
                spread[b, h, i] = p @ np.abs(v[g, :n])
                big[b, h, i] = p @ size[1][g, :n]
                reach[b, h, i] = (np.abs(q[b, h, i]) @ size[0][g, :n].T).max() * scale
    return o, lse, spread, reach, big
