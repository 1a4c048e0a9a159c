"""The cases on which the operators of the 4-bit paged cache are measured: the
write that quantises K and V rows, reading rows back, and the attention of a
decode step over the cache.

A row of d components is held in groups of ``group`` adjacent ones: codes 0 .. 15,
two to a byte (component 2i in the low half of byte i), and one 32-bit word per
group with the scale s (bf16) in its high half and the zero z (a whole number in
fp16) in its low half; the value is s (c - z).

``run`` computes a case in its plain form (elementary torch operations, 32 bits,
rounded once at the end) or, with ``own`` set, through the framework's calls.
``exact`` computes it from the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step's tokens into blocks of 16, as many heads as the fp16 decode workload: latency
        dict(name="append_step", op="append", runs=128, run=1, Hkv=40, d=128, group=32, bs=16, dtype="fp16"),
        # prompts of ragged lengths into blocks of 64
        dict(name="append_prompts", op="append", runs=13, run=631, Hkv=8, d=128, group=64, bs=64, dtype="bf16"),
        # a batch of long prompts with wide heads
        dict(name="append_long", op="append", runs=8, run=5001, Hkv=8, d=256, group=32, bs=32, dtype="bf16"),
        # the shared prefix of one conversation, read back for its next prompt: latency
        dict(name="read_one", op="read", B=1, Hkv=8, d=128, group=32, bs=16, longest=777, first=0, dtype="bf16"),
        # prefixes of ragged lengths, read back from some token on
        dict(name="read_prefixes", op="read", B=13, Hkv=8, d=128, group=64, bs=64, longest=8191, first=100,
             dtype="fp16"),
        # one short request: latency
        dict(name="decode_one", op="decode", B=1, H=32, Hkv=8, Sq=1, d=128, group=32, bs=16, longest=1000,
             mask="causal", dtype="bf16"),
        # the fp16 decode workload: 128 requests of up to 2,048 tokens, one row per K/V head
        dict(name="decode_h40", op="decode", B=128, H=40, Hkv=40, Sq=1, d=128, group=32, bs=16, longest=2048,
             mask="causal", dtype="fp16"),
        # the bf16 decode workload with four query heads per K/V head
        dict(name="decode_kv8", op="decode", B=64, H=32, Hkv=8, Sq=1, d=128, group=32, bs=64, longest=8192,
             mask="causal", dtype="bf16"),
        # the same in the smaller format
        dict(name="decode_kv8_g64", op="decode", B=64, H=32, Hkv=8, Sq=1, d=128, group=64, bs=64, longest=8192,
             mask="causal", dtype="bf16"),
        # one request over a long document
        dict(name="decode_long", op="decode", B=1, H=64, Hkv=8, Sq=1, d=128, group=64, bs=128, longest=131071,
             mask="none", dtype="bf16"),
        # small heads, eight query heads to each K/V head
        dict(name="decode_d64", op="decode", B=32, H=64, Hkv=8, Sq=1, d=64, group=32, bs=32, longest=8192,
             mask="causal", dtype="fp16"),
        # checking drafts of five tokens at d = 256, forty rows per K/V head
        dict(name="decode_drafts", op="decode", B=16, H=32, Hkv=4, Sq=5, d=256, group=32, bs=32, longest=4095,
             mask="causal", dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "decode"])
    d, group = rng.choice([64, 128, 256]), rng.choice([32, 64])
    bs, dtype = rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "fp16"])
    if op == "append":
        tokens = _log(rng, 1, 40000)
        run = min(tokens, _log(rng, 1, 5000))
        return dict(op=op, runs=max(1, tokens // run), run=run, Hkv=rng.choice([1, 2, 5, 8]), d=d, group=group,
                    bs=bs, dtype=dtype)
    if op == "read":
        longest = _log(rng, 1, 30000)
        Hkv = rng.choice([1, 2, 5, 8])
        return dict(op=op, B=max(1, min(13, int(1e8 / (longest * Hkv * d)), _log(rng, 1, 13))), Hkv=Hkv, d=d,
                    group=group, bs=bs, longest=longest, first=min(longest - 1, rng.choice([0, 0, 1, 100])), dtype=dtype)
    Hkv = rng.choice([1, 2, 4, 5, 8])
    G = rng.choice([1, 1, 2, 4, 7, 8])
    Sq = rng.choice([1, 1, 1, 2, 3, 5])
    longest = _log(rng, Sq, 131071)
    most = 3e8 / (longest * Hkv * d)
    return dict(op=op, B=max(1, min(128, int(most), _log(rng, 1, 128))), H=Hkv * G, Hkv=Hkv, Sq=Sq, d=d,
                group=group, bs=bs, longest=longest, mask=rng.choice(["causal", "none"]), dtype=dtype)


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], the first of them hi: the same for a case whatever the seed."""
    u = (np.arange(n) * 0.6180339887498949) % 1.0
    return np.maximum(lo, hi - np.floor(u * (hi - lo + 1)).astype(np.int64))


def _lens(c):
    return _spread(c["B"], max(c.get("Sq", 1), c["longest"] // 8), c["longest"])


def work(c):
    row = 2 * c["Hkv"] * (c["d"] // 2 + 4 * (c["d"] // c["group"]))  # bytes of a token in the cache
    wide = 4 * c["Hkv"] * c["d"]                                     # and in 16 bits
    if c["op"] == "append":
        tokens = c["runs"] * c["run"]
        return {"bytes": tokens * (row + wide + 4), "flops": 4 * tokens * wide // 2}
    lens = _lens(c)
    blocks = int((-(-lens // c["bs"])).sum())
    if c["op"] == "read":
        tokens = int(np.maximum(lens - c["first"], 0).sum())
        return {"bytes": tokens * (row + wide) + 4 * blocks + 8 * c["B"], "flops": tokens * wide}
    keys, rows = int(lens.sum()), c["B"] * c["H"] * c["Sq"]
    return {"bytes": keys * row + 4 * blocks + 4 * c["B"] + 4 * rows * c["d"] + 4 * rows,
            "flops": 4 * keys * c["H"] * c["Sq"] * c["d"]}


# ---------------------------------------------------------------- inputs

class State:
    pass


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _codes(shape, g):
    """Packed codes spread as those of groups of normal values are."""
    c = (torch.randn((*shape, 2), device="cuda", generator=g) * 3.4 + 7.5).round_().clamp_(0, 15).to(torch.uint8)
    return c[..., 0] | (c[..., 1] << 4)


def _words(shape, g):
    """Scale and zero of each group: sizes differ from token to token, zeros lie about the middle, some far off."""
    s = torch.exp2(torch.randn(shape, device="cuda", generator=g) * 0.5 - 2.0).to(torch.bfloat16)
    z = torch.randn(shape, device="cuda", generator=g)
    z = torch.where(torch.rand(shape, device="cuda", generator=g) < 0.02, 20.0 * z, z)
    return _pack_words(s, torch.round(7.5 + z).half())


def _pack_words(s, z):
    return (s.view(torch.int16).int() << 16) | (z.view(torch.int16).int() & 0xFFFF)


def _cache(s, pool, c, g):
    Hkv, d, bs = c["Hkv"], c["d"], c["bs"]
    s.k_cache, s.v_cache = _codes((pool, Hkv, bs, d // 2), g), _codes((pool, Hkv, bs, d // 2), g)
    s.k_scale, s.v_scale = (_words((pool, Hkv, bs, d // c["group"]), g) for _ in range(2))


def _requests(s, c, g):
    lens = _lens(c)
    need = -(-lens // c["bs"])
    M = int(need.max())
    pool = int(need.sum()) + 8
    perm = torch.randperm(pool, device="cuda", generator=g).int()
    n = torch.arange(M, device="cuda")[None]
    need_t = torch.from_numpy(need).cuda()[:, None]
    at = torch.cumsum(need_t, 0) - need_t + n
    s.table = torch.where(n < need_t, perm[at.clamp(max=pool - 1)], torch.full_like(perm[:1], -1)).contiguous()
    s.seq_lens = torch.from_numpy(lens).int().cuda()
    s.longest = int(lens.max())
    _cache(s, pool, c, g)


def _prepare_append(s, c, g):
    runs, run, Hkv, d, bs = (c[k] for k in ("runs", "run", "Hkv", "d", "bs"))
    per = -(-run // bs) + 1
    blocks = runs * per + 3
    # keys and values of a packed projection; tokens differ in size, some channels of the keys are far from 0
    x = torch.randn(runs * run, 2 * Hkv, d, device="cuda", generator=g)
    x = x * torch.exp2(torch.randn(runs * run, 1, 1, device="cuda", generator=g))
    x[:, :Hkv] += 4.0 * (torch.rand(1, Hkv, d, device="cuda", generator=g) < 0.03)
    x = x.to(DTYPES[c["dtype"]])
    s.k, s.v = x[:, :Hkv], x[:, Hkv:]
    table = torch.randperm(blocks, device="cuda", generator=g)[:runs * per].view(runs, per)
    begin = torch.randint(0, bs, (runs, 1), device="cuda", generator=g)
    pos = begin + torch.arange(run, device="cuda")[None]
    s.slots = (torch.gather(table, 1, pos // bs) * bs + pos % bs).reshape(-1).int()
    s.slots[3::97] = -1  # padding rows
    _cache(s, blocks, c, g)


def _prepare_read(s, c, g):
    _requests(s, c, g)
    s.starts = torch.full((c["B"],), c["first"], dtype=torch.int32, device="cuda")
    s.rows = max(1, s.longest - c["first"])
    # rows in front of those of the next prompt, whose keys and values go behind them
    shape = (c["B"], c["Hkv"], s.rows + 16, c["d"])
    s.out_k, s.out_v = (torch.zeros(shape, dtype=DTYPES[c["dtype"]], device="cuda")[:, :, :s.rows] for _ in range(2))


def _prepare_decode(s, c, g):
    _requests(s, c, g)
    s.q = torch.randn(c["B"], c["H"], c["Sq"], c["d"], device="cuda", generator=g).to(DTYPES[c["dtype"]])


def prepare(c, seed):
    g = _generator(seed)
    s = State()
    {"append": _prepare_append, "read": _prepare_read, "decode": _prepare_decode}[c["op"]](s, c, g)
    s.case = c
    return s


# ---------------------------------------------------------------- one pass

def _values(codes, words):
    """The values of packed rows [..., d / 2] with their groups' words [..., d / group], in 32 bits."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    scale = words.view(torch.bfloat16)[..., 1::2].float()
    zero = words.view(torch.float16)[..., 0::2].float()
    c = c.view(*words.shape, -1)
    return (scale[..., None] * (c - zero[..., None])).flatten(-2)


def _quantised(x, group):
    """Rows as packed codes and words."""
    x = x.float().unflatten(-1, (-1, group))
    low, high = x.amin(-1), x.amax(-1)
    # (hi - lo) / 15 without overflow, no less than 2^-11 of the largest, rounded up to bf16
    # (the divisor is a tensor: by a number, the quotient would be a product with its rounded inverse)
    size = (high * 0.0625 - low * 0.0625) / torch.full_like(high, 0.9375)
    size = torch.maximum(size, torch.maximum(high.abs(), low.abs()) * 2.0 ** -11)
    bits = (size.view(torch.int32) + 0xFFFF) & -65536
    s = bits.view(torch.float32)
    some = s > 0
    n = torch.round(x / torch.where(some, s, torch.ones_like(s))[..., None])
    base = torch.where(some, n.amin(-1), torch.zeros_like(s))
    c = torch.where(some[..., None], (n - base[..., None]).clamp(max=15), torch.zeros_like(n)).to(torch.uint8)
    c = c.flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), _pack_words(s.to(torch.bfloat16), (-base).half())


def _run_append(s):
    if own:
        from exact_io_aware_30_gb300 import fa
        fa.cache_append_int4(s.k, s.v, s.slots, s.k_cache, s.v_cache, s.k_scale, s.v_scale)
    else:
        c = s.case
        live = s.slots >= 0
        slots = s.slots.long()[live]
        block, at = slots // c["bs"], slots % c["bs"]
        for x, cache, scale in ((s.k, s.k_cache, s.k_scale), (s.v, s.v_cache, s.v_scale)):
            codes, words = _quantised(x[live], c["group"])
            cache[block, :, at] = codes
            scale[block, :, at] = words
    # the format fixes every bit: codes as whole numbers, equal or not; the words as
    # the scales and zeros they hold (views)
    scales = {n: w.view(torch.bfloat16)[..., 1::2] for n, w in (("k_scale", s.k_scale), ("v_scale", s.v_scale))}
    zeros = {n: w.view(torch.float16)[..., 0::2] for n, w in (("k_zero", s.k_scale), ("v_zero", s.v_scale))}
    return {"k": s.k_cache, "v": s.v_cache, **scales, **zeros}


def _gathered(cache, words, table):
    """The cached rows of each request in order, [B, Hkv, M * bs, d] in 32 bits."""
    at = table.long().clamp(min=0)
    x = _values(cache[at], words[at])
    B, M, Hkv, bs, d = x.shape
    return x.transpose(1, 2).reshape(B, Hkv, M * bs, d)


def _run_read(s):
    if own:
        from exact_io_aware_30_gb300 import fa
        return fa.cache_read_int4(s.k_cache, s.v_cache, s.k_scale, s.v_scale, s.table, s.seq_lens, s.rows,
                                  starts=s.starts, out_k=s.out_k, out_v=s.out_v)
    pos = s.starts[:, None].long() + torch.arange(s.rows, device="cuda")
    live = (pos < s.seq_lens[:, None])[:, None, :, None]
    for out, cache, words in ((s.out_k, s.k_cache, s.k_scale), (s.out_v, s.v_cache, s.v_scale)):
        x = _gathered(cache, words, s.table)
        B, Hkv, n, d = x.shape
        x = torch.gather(x, 2, pos.clamp(max=n - 1)[:, None, :, None].expand(B, Hkv, s.rows, d))
        out.copy_(torch.where(live, x.to(out.dtype), out))
    return s.out_k, s.out_v


def _run_decode(s):
    c = s.case
    if own:
        from exact_io_aware_30_gb300 import fa
        return fa.decode_paged_int4(s.q, s.k_cache, s.v_cache, s.k_scale, s.v_scale, s.table, s.seq_lens,
                                    s.longest, mask=c["mask"])
    B, H, Hkv, Sq, d = (c[k] for k in ("B", "H", "Hkv", "Sq", "d"))
    k, v = _gathered(s.k_cache, s.k_scale, s.table), _gathered(s.v_cache, s.v_scale, s.table)
    q = s.q.float().view(B, Hkv, (H // Hkv) * Sq, d)
    keys = torch.arange(k.shape[2], device="cuda")
    lens = s.seq_lens.long()[:, None]
    last = lens - 1 if c["mask"] == "none" else lens - Sq + torch.arange(H // Hkv * Sq, device="cuda") % Sq
    seen = (keys <= last[..., None])[:, None]
    x = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    x = torch.where(seen, x, torch.full_like(x[:1, :1, :1, :1], -math.inf))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / total
    return o.view(B, H, Sq, d).to(s.q.dtype), (top + torch.log(total)).view(B, H, Sq)


def run(s):
    return {"append": _run_append, "read": _run_read, "decode": _run_decode}[s.case["op"]](s)


# ---------------------------------------------------------------- 64 bits

def _exact_values(codes, words, group):
    """Rows of values in 64 bits, from the bits of the format."""
    d = codes.shape[-1] * 2
    x = torch.empty(*codes.shape[:-1], d, dtype=torch.float64, device=codes.device)
    x[..., 0::2], x[..., 1::2] = (codes % 16).double(), (codes // 16).double()
    high = (words & -65536).view(torch.float32).double()
    low = (words & 0xFFFF).to(torch.int16).view(torch.float16).double()
    for g in range(d // group):
        part = slice(g * group, (g + 1) * group)
        x[..., part] = (x[..., part] - low[..., g:g + 1]) * high[..., g:g + 1]
    return x


def _bf16_at_least(x):
    """The smallest bf16 that is not below x >= 0 (both in 64 bits)."""
    exponent = torch.frexp(x).exponent.long()
    unit = (((exponent - 8).clamp(min=-133) + 1023) << 52).view(torch.float64)
    return torch.ceil(x / unit) * unit


def _exact_append(s):
    c = s.case
    group, bs = c["group"], c["bs"]
    t = torch.nonzero(s.slots >= 0).flatten()
    slot = s.slots[t].long()
    got = {}
    for name, x, cache, words in (("k", s.k, s.k_cache, s.k_scale), ("v", s.v, s.v_cache, s.v_scale)):
        codes = cache.clone()
        scale = (words & -65536).view(torch.float32).double()
        zero = (words & 0xFFFF).to(torch.int16).view(torch.float16).double()
        rows = x[t].double()
        whole = torch.zeros_like(rows)
        for g in range(c["d"] // group):
            part = rows[..., g * group:(g + 1) * group]
            low, high = part.min(-1).values, part.max(-1).values
            # the two steps that the format takes in fp32: the difference, and the quotient
            wide = ((high - low).float().double() / 15.0).float().double()
            size = _bf16_at_least(torch.maximum(wide, part.abs().max(-1).values / 2048.0))
            safe = torch.where(size > 0, size, torch.ones_like(size))
            n = torch.round(part / safe[..., None])
            base = n.min(-1).values
            whole[..., g * group:(g + 1) * group] = (n - base[..., None]).clamp(max=15.0)
            scale[slot // bs, :, slot % bs, g] = size
            zero[slot // bs, :, slot % bs, g] = -base
        pairs = whole.view(*whole.shape[:-1], -1, 2)
        codes[slot // bs, :, slot % bs] = (pairs[..., 0] + 16.0 * pairs[..., 1]).to(torch.uint8)
        got[name], got[name + "_scale"], got[name + "_zero"] = codes, scale, zero
    return {n: got[n] for n in ("k", "v", "k_scale", "v_scale", "k_zero", "v_zero")}


def _request_rows(s, b, L, cache, words):
    blocks = s.table[b, :-(-L // s.case["bs"])].long()
    x = _exact_values(cache[blocks], words[blocks], s.case["group"])
    return x.transpose(0, 1).flatten(1, 2)[:, :L]


def _exact_read(s):
    outs = []
    for out, cache, words in ((s.out_k, s.k_cache, s.k_scale), (s.out_v, s.v_cache, s.v_scale)):
        y = out.double()
        for b, L in enumerate(s.seq_lens.tolist()):
            first = int(s.starts[b])
            if L > first:
                y[b, :, :L - first] = _request_rows(s, b, L, cache, words)[:, first:]
        outs.append(y)
    return tuple(outs)


def _exact_decode(s):
    c = s.case
    H, Hkv, Sq, d = (c[k] for k in ("H", "Hkv", "Sq", "d"))
    outs, logs = [], []
    for b, L in enumerate(s.seq_lens.tolist()):
        k, v = _request_rows(s, b, L, s.k_cache, s.k_scale), _request_rows(s, b, L, s.v_cache, s.v_scale)
        q = s.q[b].double().view(Hkv, H // Hkv, Sq, d)
        x = torch.einsum("hgid,hjd->hgij", q, k) / math.sqrt(d)
        if c["mask"] == "causal":
            i, j = torch.arange(Sq, device="cuda")[:, None], torch.arange(L, device="cuda")
            x = x.masked_fill(j > L - Sq + i, -math.inf)
        log = torch.logsumexp(x, -1)
        outs.append(torch.einsum("hgij,hjd->hgid", torch.exp(x - log[..., None]), v).reshape(H, Sq, d))
        logs.append(log.reshape(H, Sq))
    return torch.stack(outs), torch.stack(logs)


def exact(c, seed):
    s = prepare(c, seed)
    return {"append": _exact_append, "read": _exact_read, "decode": _exact_decode}[c["op"]](s)
