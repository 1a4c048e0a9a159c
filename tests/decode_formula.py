"""Attention over the 8-bit paged cache by its formula in 64 bits, with torch on
the tensors' own device (large problems; tests/step_reference.py has it one
element at a time), and the bound on the kernel's error."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def _tokens(codes, scale, blocks, n):
    """The first n tokens of the listed blocks, [Hkv, n, d] codes and [Hkv, n] scales, in 64 bits."""
    ok = (blocks >= 0) & (blocks < codes.shape[0])
    at = torch.where(ok, blocks, torch.zeros_like(blocks)).long()
    x = codes.view(torch.uint8)[at].view(torch.float8_e4m3fn).double()  # [blocks, Hkv, bs, d]
    s = scale[at].double()
    x = torch.where(ok[:, None, None, None], x, torch.zeros_like(x))
    s = torch.where(ok[:, None], s, torch.zeros_like(s))
    bs = codes.shape[2]
    return x.transpose(0, 1).flatten(1, 2)[:, :n], s.transpose(0, 1).repeat_interleave(bs, 1)[:, :n]


def decode(q, kc, vc, ks, vs, table, lens, scale, mask):
    """o [B, H, Sq, d], lse [B, H, Sq] and the pieces of the bound, in 64 bits: spread = sum of p |v|;
    reach = a row's largest sum of |q k| scale; rest = over tiles of 128 keys, the largest p |vs| of the
    tile and its two neighbours times the sum of the tile's |codes|; small = what q's components that are
    not exact can add to a score, in units of the row's largest component."""
    B, H, Sq, d = q.shape
    Hkv, bs = kc.shape[1], kc.shape[2]
    G = H // Hkv
    f64 = dict(dtype=torch.float64, device=q.device)
    o, spread, rest = (torch.zeros(B, H, Sq, d, **f64) for _ in range(3))
    lse, reach, small = (torch.full((B, H, Sq), x, **f64) for x in (-math.inf, 0.0, 0.0))
    for b in range(B):
        L = int(lens[b])
        if L == 0:
            continue
        blocks = table[b, :-(-L // bs)]
        k, ksj = _tokens(kc, ks, blocks, L)
        vcode, vsj = _tokens(vc, vs, blocks, L)
        k, v = k * ksj[..., None], vcode * vsj[..., None]
        qb = q[b].double().view(Hkv, G * Sq, d)
        x = qb @ k.transpose(1, 2) * scale
        size = qb.abs() @ k.abs().transpose(1, 2) * scale
        top = qb.abs().amax(-1, keepdim=True)
        inexact = torch.where((qb != 0) & (qb.abs() < top * 2.0 ** -13), top, torch.zeros_like(qb))
        off = inexact @ k.abs().transpose(1, 2) * scale
        seen = torch.ones(Sq, L, dtype=torch.bool, device=q.device)
        if mask == "causal":
            i, j = torch.arange(Sq, device=q.device)[:, None], torch.arange(L, device=q.device)
            seen = j <= L - Sq + i
        seen = seen.repeat(G, 1)[None]
        x = torch.where(seen, x, torch.full_like(x, -math.inf))
        l = torch.logsumexp(x, -1)
        p = torch.where(seen, torch.exp(x - torch.where(torch.isneginf(l), torch.zeros_like(l), l)[..., None]),
                        torch.zeros_like(x))
        rows = lambda t: t.reshape(H, Sq, *t.shape[2:])
        o[b], spread[b], lse[b] = rows(p @ v), rows(p @ v.abs()), rows(l)
        reach[b] = rows(torch.where(seen, size, torch.zeros_like(size)).amax(-1))
        small[b] = rows(torch.where(seen, off, torch.zeros_like(off)).amax(-1))
        tiles = -(-L // 128)
        pad = lambda t: torch.nn.functional.pad(t, (0, tiles * 128 - L))
        prod = pad(p * vsj.abs()[:, None]).view(Hkv, G * Sq, tiles, 128).amax(-1)
        wide = torch.nn.functional.max_pool1d(prod, 3, 1, 1)
        codes = pad(vcode.abs().transpose(1, 2)).view(Hkv, d, tiles, 128).sum(-1)
        rest[b] = rows(wide @ codes.transpose(1, 2))
    return o, lse, spread, reach, rest, small


def check(got, q, kc, vc, ks, vs, table, lens, scale, mask, rows=None):
    """Scores: a dot of at most 256 exact products in fp32, 2^-18 of the sum of their sizes, a q
    component below 2^-13 of its row's largest off by 2^-21 of that, and the few steps of exponent
    and logarithm.  Weights: what P V takes is a weight times its block's scale, rounded to 16 bits
    with at most four rows per K/V head, else to 8 bits (bf16: fp16's 11, then two parts of 4) or 11
    (fp16), half a step each, or to 2^-20 of the largest such product of the step's keys (at most 256, so
    within a tile and its neighbours).  fp32 sums: 2^-16 of sum p |v| over the lengths here.  O is
    rounded once.  `rows`: rows per K/V head of the call, where q is a part of it."""
    want, want_lse, spread, reach, rest, small = decode(q, kc, vc, ks, vs, table, lens, scale, mask)
    o, lse = got[0].double(), got[1].double()
    none = torch.isneginf(want_lse)
    assert torch.equal(torch.isneginf(lse), none) and bool((o[none] == 0).all())
    zero = torch.zeros_like(want_lse)
    lse, want_lse = torch.where(none, zero, lse), torch.where(none, zero, want_lse)
    tol = 2.0 ** -18 * reach + 2.0 ** -21 * small + 2.0 ** -20 * (1 + want_lse.abs())
    off = (lse - want_lse).abs()
    assert bool((off <= tol).all()), float((off / tol).max())
    rows = rows or q.shape[1] // kc.shape[1] * q.shape[2]
    weight = 2.0 ** -16 if rows <= 4 else 2.0 ** -11 + (2.0 ** -8 if q.dtype == torch.bfloat16 else 0.0)
    bound = (weight + 2.0 ** -16 + 2 * tol[..., None]) * spread + HALF_STEP[q.dtype] * want.abs() + 2.0 ** -20 * rest + \
        2.0 ** -24
    off = (o - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())


def problem(B, H, Hkv, Sq, d, bs, lens, dtype, seed, max_blocks=None, vs=None, device="cuda"):
    """Random q, caches of normal codes, scales 2^-8 .. 2^-6, scattered blocks; NaN codes behind each
    request's end and NaN scales in the blocks nobody has."""
    g = torch.Generator(device=device).manual_seed(seed)
    lens = torch.as_tensor(lens, dtype=torch.int32)
    need = (lens + bs - 1) // bs
    M = max(1, int(need.max())) if max_blocks is None else max_blocks
    pool = int(need.sum()) + 3
    perm = torch.randperm(pool, device=device, generator=g).int()
    table = torch.full((B, M), -1, dtype=torch.int32, device=device)
    at = 0
    rnd = lambda *s: torch.randn(*s, device=device, generator=g)
    kc, vc = ((rnd(pool, Hkv, bs, d) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2))
    scales = [torch.exp2(torch.randint(-8, -5, (pool, Hkv), device=device, generator=g).float()) for _ in range(2)]
    for b in range(B):
        n, L = int(need[b]), int(lens[b])
        table[b, :n] = perm[at:at + n]
        at += n
        if L % bs:
            last = int(table[b, n - 1])
            kc[last, :, L % bs:] = 0x7F
            vc[last, :, L % bs:] = 0xFF
    unused = perm[at:].long()
    for c, s in zip((kc, vc), scales):
        c[unused] = 0x7F
        s[unused] = math.nan
    q = rnd(B, H, Sq, d).to(dtype)
    return [q, kc, vc, scales[0], scales[1], table, lens.to(device)]
