"""The cases on which the decode-step operators are measured: block tables and
slot maps, rotary positions, the write into the 8-bit paged cache, and the
attention that reads that cache.

``run`` computes a case in its plain form (elementary torch operations, 32 bits,
rounded once at the end) or, with ``own`` set, through the framework's calls.
``exact`` computes it from the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3_MAX = 448.0


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step of 64 requests with grouped heads: latency
        dict(name="rope_step", op="rope", B=64, S=1, H=32, Hkv=8, d=128, rot=128, layout="half",
             scaling="none", dtype="bf16", far=8192, packed=True, backward=False),
        # a training forward of 8k tokens, read out of the packed projection's output
        dict(name="rope_8k", op="rope", B=1, S=8192, H=32, Hkv=32, d=128, rot=128, layout="half",
             scaling="none", dtype="fp16", far=0, packed=True, backward=False),
        # the gradient of a part-of-the-head rotation in a training step
        dict(name="rope_bwd_part", op="rope", B=4, S=2048, H=16, Hkv=16, d=128, rot=64,
             layout="interleaved", scaling="none", dtype="bf16", far=0, packed=False, backward=True),
        # a long prompt's chunk at far positions with scaled frequencies, in fp32, odd length
        dict(name="rope_far_fp32", op="rope", B=1, S=4097, H=8, Hkv=2, d=256, rot=256, layout="half",
             scaling="by_parts", dtype="fp32", far=1000000, packed=False, backward=False),
        # one decode step: every request grows by one token
        dict(name="update_step", op="update", B=64, M=128, bs=64, T=64, grow=1, mixed=False),
        # prompts, decode steps, rejected drafts and finished requests in one step
        dict(name="update_mixed", op="update", B=513, M=256, bs=16, T=65536, grow=512, mixed=True),
        # one decode step's tokens into blocks of 16, as many heads as the fp16 decode workload
        dict(name="append_step", op="append", runs=128, run=1, Hkv=40, d=128, bs=16, dtype="fp16"),
        # prompts of ragged lengths into blocks of 64
        dict(name="append_prompts", op="append", runs=13, run=631, Hkv=8, d=128, bs=64, dtype="bf16"),
        # one short request: latency
        dict(name="decode_one", op="decode", B=1, H=32, Hkv=8, Sq=1, d=128, bs=16, longest=1000,
             mask="causal", dtype="bf16"),
        # the fp16 decode workload: 128 requests of up to 2,048 tokens, one row per K/V head
        dict(name="decode_h40", op="decode", B=128, H=40, Hkv=40, Sq=1, d=128, bs=16, longest=2048,
             mask="causal", dtype="fp16"),
        # the bf16 decode workload with four query heads per K/V head
        dict(name="decode_kv8", op="decode", B=64, H=32, Hkv=8, Sq=1, d=128, bs=64, longest=8192,
             mask="causal", dtype="bf16"),
        # checking drafts of five tokens at d = 256, forty rows per K/V head
        dict(name="decode_drafts", op="decode", B=16, H=32, Hkv=4, Sq=5, d=256, bs=32, longest=4095,
             mask="causal", dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "update", "append", "decode", "decode"])
    if op == "rope":
        d = rng.choice([64, 80, 128, 256])
        H = rng.choice([1, 5, 8, 16, 32])
        Hkv = rng.choice([h for h in (1, 2, 4, 5, 8, 16, 32) if H % h == 0])
        tokens = _log(rng, 1, 8192)
        B = rng.choice([1, 1, 2, 3, 7])
        return dict(op=op, B=B, S=max(1, tokens // B), H=H, Hkv=Hkv, d=d,
                    rot=rng.choice([d, d, d // 2, d // 4 + 2 - d // 4 % 2]),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "by_parts"]),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), far=rng.choice([0, 8192, 1000000]),
                    packed=rng.random() < 0.5, backward=rng.random() < 0.4)
    if op == "update":
        B = _log(rng, 1, 2000)
        mixed = rng.random() < 0.6
        grow = _log(rng, 2, 300) if mixed else rng.choice([1, 1, 2, 5])
        bs = rng.choice([16, 32, 64, 128])
        return dict(op=op, B=B, M=2 + _log(rng, 4096, 16384) // bs, bs=bs,
                    T=max(1, min(65536, B * grow - rng.randrange(0, 3))), grow=grow, mixed=mixed)
    if op == "append":
        tokens = _log(rng, 1, 8192)
        run = min(tokens, _log(rng, 1, 700))
        return dict(op=op, runs=max(1, tokens // run), run=run, Hkv=rng.choice([1, 2, 5, 8, 16]),
                    d=rng.choice([64, 128, 256]), bs=rng.choice([16, 32, 64, 128]),
                    dtype=rng.choice(["bf16", "fp16"]))
    Hkv = rng.choice([1, 2, 4, 5, 8])
    G = rng.choice([1, 1, 2, 4, 7, 8])
    Sq = rng.choice([1, 1, 1, 2, 3, 5])
    d = rng.choice([64, 128, 256])
    longest = _log(rng, Sq, 100000)
    most = 3e8 / (longest * Hkv * d * 2)
    return dict(op=op, B=max(1, min(128, int(most), _log(rng, 1, 128))), H=Hkv * G, Hkv=Hkv, Sq=Sq, d=d,
                bs=rng.choice([16, 32, 64, 128]), longest=longest, mask=rng.choice(["causal", "none"]),
                dtype=rng.choice(["bf16", "fp16"]))


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], the first of them hi: the same for a case whatever the seed."""
    u = (np.arange(n) * 0.6180339887498949) % 1.0
    return np.maximum(lo, hi - np.floor(u * (hi - lo + 1)).astype(np.int64))


def work(c):
    if c["op"] == "rope":
        size = 4 if c["dtype"] == "fp32" else 2
        n = c["B"] * c["S"] * (c["H"] + c["Hkv"])
        return {"bytes": 2 * n * c["d"] * size + c["B"] * c["S"] * 4, "flops": 3 * n * c["rot"]}
    if c["op"] == "update":
        delta = _deltas(c)
        grown = int(np.maximum(delta, 0).sum())
        return {"bytes": 16 * c["B"] + 8 * c["T"] + 8 * (grown // c["bs"]) + 16, "flops": 0}
    if c["op"] == "append":
        tokens, blocks = c["runs"] * c["run"], c["runs"] * (-(-c["run"] // c["bs"]))
        return {"bytes": 6 * tokens * c["Hkv"] * c["d"] + 8 * blocks * c["Hkv"] + 4 * tokens,
                "flops": 4 * tokens * c["Hkv"] * c["d"]}
    lens = _spread(c["B"], max(c["Sq"], c["longest"] // 8), c["longest"])
    keys, blocks = int(lens.sum()), int((-(-lens // c["bs"])).sum())
    rows = c["B"] * c["H"] * c["Sq"]
    return {"bytes": 2 * keys * c["Hkv"] * c["d"] + 8 * blocks * c["Hkv"] + 4 * blocks + 4 * rows * c["d"] + 4 * rows,
            "flops": 4 * keys * c["H"] * c["Sq"] * c["d"]}


# ---------------------------------------------------------------- inputs

class State:
    pass


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


SCALED = {"none": {}, "linear": dict(factor=4.0), "ntk": dict(factor=4.0),
          "by_parts": dict(factor=16.0, original_length=4096)}


def _frequencies(rot, scaling):
    """Radians per position of each pair and the amplitude, in 64 bits."""
    i = np.arange(rot // 2, dtype=np.float64)
    base = 10000.0
    if scaling == "ntk" and rot > 2:
        base = base * 4.0 ** (rot / (rot - 2.0))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / 4.0, 1.0
    if scaling == "by_parts":
        turns = 4096 * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return f * (keep + (1.0 - keep) / 16.0), 0.1 * math.log(16.0) + 1.0
    return f, 1.0


def _prepare_rope(c, g):
    s = State()
    B, S, H, Hkv, d = (c[k] for k in ("B", "S", "H", "Hkv", "d"))
    dt = DTYPES[c["dtype"]]
    if c["packed"]:  # [B, S, (q heads, k heads, v heads), d], as one projection writes it
        x = torch.randn(B, S, H + 2 * Hkv, d, device="cuda", generator=g).to(dt)
        s.q, s.k = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hkv].transpose(1, 2)
    else:
        s.q = torch.randn(B, H, S, d, device="cuda", generator=g).to(dt)
        s.k = torch.randn(B, Hkv, S, d, device="cuda", generator=g).to(dt)
    start = torch.randint(0, c["far"] + 1, (B, 1), device="cuda", generator=g)
    s.positions = (start + torch.arange(S, device="cuda")[None]).int()
    f, s.amplitude = _frequencies(c["rot"], c["scaling"])
    s.f = torch.from_numpy(f).cuda()
    if own:
        from exact_io_aware_30_gb300 import fa
        s.plan = fa.rope_plan(c["rot"], base=10000.0, scaling=c["scaling"], device="cuda",
                              **SCALED[c["scaling"]])
    return s


def _deltas(c):
    if not c["mixed"]:
        delta = np.full(c["B"], c["grow"], np.int64)
        delta[5::17] = 0  # padding rows of a captured batch
        return delta
    delta = np.minimum(c["grow"], 1 + _spread(c["B"], 0, c["grow"]) ** 2 // c["grow"])
    delta[1::3] = 1
    delta[2::7] = -2    # rejected drafts
    delta[4::11] = -(1 << 30)  # finished
    return delta


def _prepare_update(c, g):
    s = State()
    B, M, bs = c["B"], c["M"], c["bs"]
    s.seq_lens = torch.randint(0, M * bs - c["grow"] + 1, (B,), device="cuda", generator=g).int()
    s.delta = torch.from_numpy(_deltas(c)).int().cuda()
    blocks = (s.seq_lens.long() + bs - 1) // bs
    pool = B * M
    perm = torch.randperm(pool, device="cuda", generator=g).int()
    s.table = perm.view(B, M).clone()
    live = torch.arange(M, device="cuda")[None] < blocks[:, None]
    free = s.table[~live]
    # the ring holds the free blocks from some place on, round its end
    s.ring = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
    head = torch.randint(0, pool, (1,), device="cuda", generator=g)
    s.ring[(head + torch.arange(free.numel(), device="cuda")) % pool] = free
    s.table[~live] = -1
    s.ring_state = torch.cat([head, torch.full_like(head, free.numel())]).int()
    s.out = dict(seq_lens_out=torch.empty_like(s.seq_lens), ring_state_out=torch.empty_like(s.ring_state),
                 slot_map=torch.empty(c["T"], dtype=torch.int32, device="cuda"),
                 positions=torch.empty(c["T"], dtype=torch.int32, device="cuda"),
                 status=torch.empty_like(s.seq_lens))
    return s


def _codes(shape, g):
    """e4m3 codes of normal values whose largest are near the type's largest."""
    return (torch.randn(shape, device="cuda", generator=g) * 100).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _scales(shape, g):
    return torch.exp2(torch.randint(-8, -5, shape, device="cuda", generator=g).float())


def _prepare_append(c, g):
    s = State()
    runs, run, Hkv, d, bs = (c[k] for k in ("runs", "run", "Hkv", "d", "bs"))
    per = -(-run // bs) + 1
    blocks = runs * per + 3
    dt = DTYPES[c["dtype"]]
    # keys and values of a packed projection; tokens differ in size
    x = torch.randn(runs * run, 2 * Hkv, d, device="cuda", generator=g)
    x = (x * torch.exp2(torch.randn(runs * run, 1, 1, device="cuda", generator=g))).to(dt)
    s.k, s.v = x[:, :Hkv], x[:, Hkv:]
    table = torch.randperm(blocks, device="cuda", generator=g)[:runs * per].view(runs, per)
    begin = torch.randint(0, bs, (runs, 1), device="cuda", generator=g)
    pos = begin + torch.arange(run, device="cuda")[None]
    slots = torch.gather(table, 1, pos // bs) * bs + pos % bs
    s.slots = slots.reshape(-1).int()
    s.slots[3::97] = -1  # padding rows
    s.k_cache, s.v_cache = _codes((blocks, Hkv, bs, d), g), _codes((blocks, Hkv, bs, d), g)
    s.k_scale, s.v_scale = _scales((blocks, Hkv), g), _scales((blocks, Hkv), g)
    return s


def _prepare_decode(c, g):
    s = State()
    B, H, Hkv, Sq, d, bs = (c[k] for k in ("B", "H", "Hkv", "Sq", "d", "bs"))
    lens = _spread(B, max(Sq, c["longest"] // 8), c["longest"])
    need = -(-lens // bs)
    M = int(need.max())
    pool = int(need.sum()) + 8
    perm = torch.randperm(pool, device="cuda", generator=g).int()
    n = torch.arange(M, device="cuda")[None]
    need_t = torch.from_numpy(need).cuda()[:, None]
    at = torch.cumsum(need_t, 0) - need_t + n
    s.table = torch.where(n < need_t, perm[at.clamp(max=pool - 1)], torch.full_like(perm[:1], -1)).contiguous()
    s.seq_lens = torch.from_numpy(lens).int().cuda()
    s.longest = int(lens.max())
    s.q = torch.randn(B, H, Sq, d, device="cuda", generator=g).to(DTYPES[c["dtype"]])
    s.k_cache, s.v_cache = _codes((pool, Hkv, bs, d), g), _codes((pool, Hkv, bs, d), g)
    s.k_scale, s.v_scale = _scales((pool, Hkv), g), _scales((pool, Hkv), g)
    return s


def prepare(c, seed):
    g = _generator(seed)
    s = {"rope": _prepare_rope, "update": _prepare_update, "append": _prepare_append,
         "decode": _prepare_decode}[c["op"]](c, g)
    s.case = c
    return s


# ---------------------------------------------------------------- one pass

def _rotate_plain(x, s, sign):
    c = s.case
    rot, half = c["rot"], c["rot"] // 2
    angle = s.positions.double()[:, None, :, None] * s.f
    cos, sin = (s.amplitude * torch.cos(angle)).float(), (sign * s.amplitude * torch.sin(angle)).float()
    y = x.float()
    if c["layout"] == "half":
        a, b = y[..., :half], y[..., half:rot]
        r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([r, y[..., rot:]], -1).to(x.dtype)


def _run_rope(s):
    c = s.case
    if own:
        from exact_io_aware_30_gb300 import fa
        call = fa.rope_backward if c["backward"] else fa.rope
        return call(s.q, s.k, s.plan, positions=s.positions, layout=c["layout"])
    sign = -1.0 if c["backward"] else 1.0
    return _rotate_plain(s.q, s, sign), _rotate_plain(s.k, s, sign)


def _update_plain(s):
    c = s.case
    M, bs, T = c["M"], c["bs"], c["T"]
    C = s.ring.numel()
    head, count = s.ring_state[0].long(), s.ring_state[1].long()
    old, delta = s.seq_lens.long().clamp(0, M * bs), s.delta.long()
    add = delta.clamp(min=0)
    upto = torch.cumsum(add, 0)
    first = upto - add
    have = (old + bs - 1) // bs
    long, wide = old + add > M * bs, upto > T
    need = torch.where((add > 0) & ~long & ~wide, (old + add + bs - 1) // bs - have, torch.zeros_like(have))
    start = torch.cumsum(need, 0) - need
    short = (need > 0) & (start + need > count)
    zero = torch.zeros_like(have)
    status = torch.where(add > 0, torch.where(long, zero + 2, torch.where(wide, zero + 3, short.long())), zero)
    new = torch.where(status == 0, (old + delta).clamp(min=0), old)
    need = torch.where(short, zero, need)
    used = need.sum()
    n = torch.arange(M, device="cuda")[None]
    j = n - have[:, None]
    table = torch.where((j >= 0) & (j < need[:, None]), s.ring[(head + start[:, None] + j) % C], s.table)
    keep = (new + bs - 1) // bs
    gone = (have - keep).clamp(min=0)
    order = (torch.cumsum(gone, 0) - gone)[:, None] + n - keep[:, None]
    push = (n >= keep[:, None]) & (n < have[:, None]) & (order < C - count)
    at = torch.where(push, (head + count + order) % C, torch.full_like(order, C))
    ring = torch.cat([s.ring, s.ring[:1]]).scatter(0, at.reshape(-1), s.table.reshape(-1))[:C]
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(upto, t, right=True).clamp(max=c["B"] - 1)
    pos = old[b] + t - first[b]
    live = (t < upto[-1]) & (status[b] == 0)
    block = table[b, (pos // bs).clamp(0, M - 1)].long()
    live = live & (block >= 0)
    slot = torch.where(live, block * bs + pos % bs, torch.full_like(pos, -1))
    pos = torch.where(live, pos, torch.zeros_like(pos))
    state = torch.stack([(head + used) % C, count - used + push.sum()])
    return {"seq_lens": new.int(), "ring_state": state.int(), "slot_map": slot.int(), "positions": pos.int(),
            "status": status.int(), "block_table": table.int(), "free_ring": ring.int()}


def _run_update(s):
    if own:
        from exact_io_aware_30_gb300 import fa
        r = fa.paged_update(s.seq_lens, s.delta, s.table, s.ring, s.ring_state, s.case["bs"], **s.out)
        return {"seq_lens": r.seq_lens, "ring_state": r.ring_state, "slot_map": r.slot_map,
                "positions": r.positions, "status": r.status, "block_table": s.table, "free_ring": s.ring}
    return _update_plain(s)


def _append_plain(x, slots, cache, scale):
    """One of K and V: the new cache and scales (powers of two where the call sets them)."""
    blocks, Hkv, bs, d = cache.shape
    live = slots >= 0
    slots, x = slots.long()[live], x.float()[live]
    block, at = slots // bs, slots % bs
    size = x.abs().amax(-1)
    amax = torch.zeros(blocks, Hkv, device="cuda")
    amax.scatter_reduce_(0, block[:, None].expand(-1, Hkv), size, "amax")
    mantissa, exponent = torch.frexp(amax)
    exponent = (exponent - 9 + (mantissa > 0.875).int()).clamp(min=-126)
    need = torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, exponent, torch.full_like(exponent, -126)))
    touched, begun = torch.zeros(blocks, 1, device="cuda"), torch.zeros(blocks, 1, device="cuda")
    touched[block] = 1
    begun.scatter_reduce_(0, block[:, None], (at == 0).float()[:, None], "amax")
    new = torch.where(touched > 0, torch.where(begun > 0, need, torch.maximum(scale, need)), scale)
    grew = (touched > 0) & (begun == 0) & (new > scale)
    again = (cache.float() * scale[..., None, None] / new[..., None, None]).clamp(-E4M3_MAX, E4M3_MAX)
    codes = torch.where(grew[..., None, None], again.to(torch.float8_e4m3fn).view(torch.uint8), cache.view(torch.uint8))
    written = (x / new[block][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    codes[block, :, at] = written.view(torch.uint8)
    return codes.view(torch.float8_e4m3fn), new


def _run_append(s):
    if own:
        from exact_io_aware_30_gb300 import fa
        fa.cache_append_fp8(s.k, s.v, s.slots, s.k_cache, s.v_cache, s.k_scale, s.v_scale)
    else:
        k, ks = _append_plain(s.k, s.slots, s.k_cache, s.k_scale)
        v, vs = _append_plain(s.v, s.slots, s.v_cache, s.v_scale)
        s.k_cache.view(torch.uint8).copy_(k.view(torch.uint8))
        s.v_cache.view(torch.uint8).copy_(v.view(torch.uint8))
        s.k_scale.copy_(ks)
        s.v_scale.copy_(vs)
    return {"k": s.k_cache, "v": s.v_cache, "k_scale": s.k_scale, "v_scale": s.v_scale}


def _gathered(cache, scale, table):
    """The cached rows of each request in order, [B, Hkv, M * bs, d] in 32 bits."""
    at = table.long().clamp(min=0)
    x = cache.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * scale[at][..., None, None]
    B, M, Hkv, bs, d = x.shape
    return x.transpose(1, 2).reshape(B, Hkv, M * bs, d)


def _decode_plain(s):
    c = s.case
    B, H, Hkv, Sq, d = (c[k] for k in ("B", "H", "Hkv", "Sq", "d"))
    k, v = _gathered(s.k_cache, s.k_scale, s.table), _gathered(s.v_cache, s.v_scale, s.table)
    q = s.q.float().view(B, Hkv, (H // Hkv) * Sq, d)
    keys = torch.arange(k.shape[2], device="cuda")
    lens = s.seq_lens.long()[:, None]
    last = lens - 1 if c["mask"] == "none" else lens - Sq + torch.arange(H // Hkv * Sq, device="cuda") % Sq
    seen = (keys <= last[..., None])[:, None]
    v = torch.where((keys < lens)[:, None, :, None], v, torch.zeros_like(v[:1, :1, :1, :1]))
    x = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    x = torch.where(seen, x, torch.full_like(x[:1, :1, :1, :1], -math.inf))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / total
    return o.view(B, H, Sq, d).to(s.q.dtype), (top + torch.log(total)).view(B, H, Sq)


def _run_decode(s):
    if own:
        from exact_io_aware_30_gb300 import fa
        return fa.decode_paged_fp8(s.q, s.k_cache, s.v_cache, s.k_scale, s.v_scale, s.table, s.seq_lens,
                                   s.longest, mask=s.case["mask"])
    return _decode_plain(s)


def run(s):
    return {"rope": _run_rope, "update": _run_update, "append": _run_append, "decode": _run_decode}[s.case["op"]](s)


# ---------------------------------------------------------------- 64 bits

def _exact_rope(s):
    c = s.case
    sign = -1.0 if c["backward"] else 1.0
    turn = torch.polar(torch.full_like(s.f, s.amplitude), torch.zeros_like(s.f))
    turn = turn * torch.exp(1j * sign * s.positions.double()[:, None, :, None] * s.f)
    out = []
    for x in (s.q, s.k):
        y = x.double().clone()
        half = c["rot"] // 2
        first, second = (slice(0, half), slice(half, c["rot"])) if c["layout"] == "half" else \
            (slice(0, c["rot"], 2), slice(1, c["rot"], 2))
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _nearest_e4m3(x):
    """The nearest value of e4m3, ties to even, saturating."""
    exponent = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6)
    step = torch.exp2(exponent - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_append(s):
    got = {}
    slots = s.slots.cpu().numpy()
    bs = s.case["bs"]
    rows = {}
    for t, slot in enumerate(slots):
        if slot >= 0:
            rows.setdefault(int(slot) // bs, []).append((t, int(slot) % bs))
    for name, x, cache, scale in (("k", s.k, s.k_cache, s.k_scale), ("v", s.v, s.v_cache, s.v_scale)):
        values, scales, x = cache.double().clone(), scale.double().clone(), x.double()
        for block, pairs in rows.items():
            t = torch.tensor([p[0] for p in pairs], device="cuda")
            at = torch.tensor([p[1] for p in pairs], device="cuda")
            new = x[t].transpose(0, 1)  # [Hkv, n, d]
            need = torch.exp2(torch.ceil(torch.log2(new.abs().amax((1, 2)) / E4M3_MAX)))
            old = scales[block].clone()
            begun = bool((at == 0).any())
            now = need if begun else torch.maximum(old, need)
            if not begun:
                values[block] = _nearest_e4m3(values[block] * (old / now)[:, None, None])
            values[block, :, at] = _nearest_e4m3(new / now[:, None, None])
            scales[block] = now
        got[name], got[name + "_scale"] = values, scales
    return {"k": got["k"], "v": got["v"], "k_scale": got["k_scale"], "v_scale": got["v_scale"]}


def _exact_decode(s):
    c = s.case
    H, Hkv, Sq, d, bs = (c[k] for k in ("H", "Hkv", "Sq", "d", "bs"))
    outs, logs = [], []
    for b, L in enumerate(s.seq_lens.tolist()):
        blocks = s.table[b, :-(-L // bs)].long()

        def rows(cache, scale):
            x = cache[int(blocks[0]):int(blocks[0]) + 1] if blocks.numel() == 1 else \
                cache.view(torch.uint8)[blocks].view(torch.float8_e4m3fn)
            x = x.double() * scale[blocks].double()[..., None, None]
            return x.transpose(0, 1).flatten(1, 2)[:, :L]

        k, v = rows(s.k_cache, s.k_scale), rows(s.v_cache, s.v_scale)
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
    if c["op"] == "update":  # whole numbers only
        return None
    return {"rope": _exact_rope, "append": _exact_append, "decode": _exact_decode}[c["op"]](s)
