"""Plain 64-bit (or whole-number) implementations of the decode step's
operators: rotary positions, the paged cache's bookkeeping, the quantising
append and attention over the 8-bit cache.  Written from the formulas in
include/fa.h, one element at a time where that is clearest."""
import math

import numpy as np

from exact_io_aware_30_gb300 import inputs


def radians(rot, base=10000.0, scaling="none", factor=1.0, original_length=0.0, low_turns=1.0,
            high_turns=32.0):
    """Radians per position of each pair and the amplitude."""
    out = []
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f = f / factor
        elif scaling == "by_parts":
            turns = original_length * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - low_turns) / (high_turns - low_turns)))
            f = keep * f + (1 - keep) * f / factor
        out.append(f)
    return np.array(out), (0.1 * math.log(factor) + 1.0 if scaling == "by_parts" else 1.0)


def rotate(x, positions, f, amplitude, layout, sign=1.0):
    """x [B, H, S, d] float64, positions [B, S]; sign -1: the transposed map."""
    y = x.copy()
    rot = 2 * len(f)
    first = np.arange(0, rot // 2) if layout == "half" else np.arange(0, rot, 2)
    second = first + (rot // 2 if layout == "half" else 1)
    theta = positions.astype(np.float64)[:, None, :, None] * f
    c, s = amplitude * np.cos(theta), sign * amplitude * np.sin(theta)
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., first] * s + x[..., second] * c
    return y


def paged_update(seq_lens, delta, table, ring, state, bs, rows):
    """One request after another; returns new copies of everything."""
    table, ring = table.copy(), ring.copy()
    B, M = table.shape
    C = len(ring)
    head, count = int(state[0]), int(state[1])
    new, status = np.zeros(B, np.int32), np.zeros(B, np.int32)
    slot, position = np.full(rows, -1, np.int32), np.zeros(rows, np.int32)
    first = taken = asked = 0
    back = []
    for b in range(B):
        old = min(max(int(seq_lens[b]), 0), M * bs)
        have, change = -(-old // bs), int(delta[b])
        new[b] = old
        if change < 0:
            new[b] = max(old + change, 0)
            back += [int(x) for x in table[b, -(-int(new[b]) // bs):have]]
        if change > 0:
            need = -(-(old + change) // bs) - have
            if old + change > M * bs:
                status[b] = 2
            elif first + change > rows:
                status[b] = 3
            else:
                if need > 0 and asked + need > count:
                    status[b] = 1
                asked += need
            if status[b] == 0:
                for j in range(need):
                    table[b, have + j] = ring[(head + taken + j) % C]
                taken += need
                new[b] = old + change
                for i in range(change):
                    block = int(table[b, (old + i) // bs])
                    if block >= 0 and block * bs + bs <= 2 ** 31:
                        slot[first + i] = block * bs + (old + i) % bs
                        position[first + i] = old + i
            first += change
    pushed = 0
    for x in back:
        if pushed < C - count:
            ring[(head + count + pushed) % C] = x
            pushed += 1
    return dict(seq_lens=new, status=status, slot_map=slot, positions=position, block_table=table,
                free_ring=ring, ring_state=np.array([(head + taken) % C, count - taken + pushed], np.int32))


def smallest_scale(amax):
    """The smallest power of two s >= 2^-126 with amax <= 448 s."""
    s = 2.0 ** -126
    while amax > 448.0 * s:
        s *= 2.0
    return s


def append(x, slots, codes, scale, bs):
    """x [T, Hkv, d] float64 (of 16-bit values); codes [blocks, Hkv, bs, d] uint8, scale fp32."""
    codes, scale = codes.copy(), scale.copy()
    blocks, Hkv = scale.shape
    rows = {}
    for t, s in enumerate(slots):
        if 0 <= s < blocks * bs:
            rows.setdefault(int(s) // bs, {})[int(s) % bs] = t
    with np.errstate(invalid="ignore", over="ignore"):
        for block, written in rows.items():
            for h in range(Hkv):
                vals = np.concatenate([x[t, h] for t in written.values()])
                vals = np.abs(vals[np.isfinite(vals)])
                need = smallest_scale(vals.max() if vals.size else 0.0)
                old = float(scale[block, h])
                valid = old > 0 and np.isfinite(old)
                now = need if 0 in written or not valid else max(old, need)
                if 0 not in written and valid and now > old:
                    for at in range(bs):
                        if at not in written:
                            v = inputs.e4m3_bits_to_f64(codes[block, h, at])
                            again = inputs.f32_to_e4m3_bits(
                                np.float32(v.astype(np.float32) * np.float32(old)) / np.float32(now))
                            codes[block, h, at] = np.where(np.isnan(v), codes[block, h, at], again)
                for at, t in written.items():
                    v = (x[t, h].astype(np.float32) / np.float32(now)).astype(np.float64)
                    codes[block, h, at] = np.where(np.isnan(v), 0x7F, inputs.f32_to_e4m3_bits(
                        np.nan_to_num(v, nan=0.0, posinf=1e30, neginf=-1e30)))
                scale[block, h] = now
    return codes, scale


def gathered(codes, scale, table_row, n, bs):
    """The first n tokens of a request, [Hkv, n, d] float64; entries outside the pool read zeros."""
    blocks, Hkv, _, d = codes.shape
    out = np.zeros((Hkv, n, d))
    for i in range(-(-n // bs)):
        block = int(table_row[i])
        k = min(bs, n - i * bs)
        if 0 <= block < blocks:
            out[:, i * bs:i * bs + k] = inputs.e4m3_bits_to_f64(codes[block, :, :k]) * scale[block].astype(np.float64)[:, None, None]
    return out


def decode(q, kc, vc, ks, vs, table, lens, max_len, scale, mask, bs):
    """(o, lse, spread) in float64: spread [B, H, Sq, d] is the sum of p |v|, what rounding a weight
    is relative to; also the largest sum of |q k| scale of a row, [B, H, Sq]."""
    B, H, Sq, d = q.shape
    Hkv = kc.shape[1]
    o, spread = np.zeros_like(q), np.zeros_like(q)
    lse, reach = np.full((B, H, Sq), -np.inf), np.zeros((B, H, Sq))
    for b in range(B):
        L = min(max(int(lens[b]), 0), max_len)
        if L == 0:
            continue
        k, v = gathered(kc, ks, table[b], L, bs), gathered(vc, vs, table[b], L, bs)
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
                reach[b, h, i] = (np.abs(q[b, h, i]) @ np.abs(k[g, :n]).T).max() * scale
    return o, lse, spread, reach
