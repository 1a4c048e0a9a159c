"""The 4-bit paged cache on the GPU: the quantising append (fa_cache_append_int4),
reading back (fa_cache_read_int4) and attention over it (fa_decode_paged_int4),
each against the formulas in 64 bits, and a run of them as a program uses them."""
import numpy as np
import pytest

import int4_reference as ref
from exact_io_aware_30_gb300 import fa, inputs

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

U = {inputs.BF16: 2.0 ** -8, inputs.FP16: 2.0 ** -11}  # half a step of the type, relative to the value
DTYPES = {inputs.BF16: torch.bfloat16, inputs.FP16: torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from exact_io_aware_30_gb300 import build
    build.build()
    fa.load()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    assert fa.device_error() == fa.FA_OK


def _t16(bits, dtype):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(DTYPES[dtype]).cuda()


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _rows(rng, shape, dtype, kind="normal"):
    """16-bit rows as bits: sizes differ from row to row, some channels lie far from 0."""
    x = rng.standard_normal(shape) * 2.0 ** rng.integers(-3, 4, (*shape[:-1], 1))
    if kind == "offset":
        x = x * 2.0 ** -6 + rng.choice([0.0, 3.0, -100.0], (*shape[:-1], 1))
    if kind == "ties":  # values on halves of the grid
        x = rng.integers(-15, 16, shape) * 0.5
    if kind == "wide":
        top = 15.0 if dtype == inputs.FP16 else 126.0
        x = np.sign(x) * 2.0 ** rng.uniform(-top, top, shape)
    return inputs.to_bits(x.astype(np.float32), dtype)


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
@pytest.mark.parametrize("kind", ["normal", "offset", "ties", "wide"])
@pytest.mark.parametrize("T,Hkv,d,group,bs", [(1, 1, 64, 32, 16), (7, 3, 128, 32, 16), (130, 2, 256, 64, 32),
                                              (33, 5, 64, 64, 128), (300, 1, 128, 64, 64), (65, 8, 256, 32, 16)])
def test_append_is_the_format_to_the_bit(T, Hkv, d, group, bs, kind, dtype):
    rng = np.random.default_rng(T + d + group)
    blocks = -(-T // bs) + 3
    slots = rng.permutation(blocks * bs)[:T].astype(np.int32)
    slots[rng.random(T) < 0.1] = -1
    slots[rng.random(T) < 0.05] = blocks * bs  # past the pool
    kb, vb = (_rows(rng, (T, Hkv, d), dtype, kind) for _ in range(2))
    codes = [rng.integers(0, 256, (blocks, Hkv, bs, d // 2)).astype(np.uint8) for _ in range(2)]
    w = [rng.integers(-2 ** 31, 2 ** 31, (blocks, Hkv, bs, d // group)).astype(np.int32) for _ in range(2)]
    got_c, got_w = [_dev(c) for c in codes], [_dev(x) for x in w]
    # heads of a packed projection
    x = torch.empty(T, 2 * Hkv, d, dtype=DTYPES[dtype], device="cuda")
    x[:, :Hkv], x[:, Hkv:] = _t16(kb, dtype), _t16(vb, dtype)
    fa.cache_append_int4(x[:, :Hkv], x[:, Hkv:], _dev(slots), *got_c, *got_w)
    for bits, c, ww, gc, gw in zip((kb, vb), codes, w, got_c, got_w):
        want_c, want_w = ref.append(inputs.bits_to_f64(bits, dtype), slots, c, ww, bs, group)
        assert np.array_equal(gw.cpu().numpy(), want_w)
        assert np.array_equal(gc.cpu().numpy(), want_c)


@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
def test_append_constants_zeros_and_what_is_no_number(dtype):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((12, 1, 64)).astype(np.float32)
    x[0] = 0
    x[1] = 3.25
    x[2] = -1e-3
    x[3, 0, 5] = np.inf
    x[4, 0, 40] = -np.inf
    x[5, 0, 0] = np.nan
    x[6, 0, :32] = 6e4
    x[6, 0, 3] = -6e4
    x[7] = 0
    x[7, 0, 9] = 2.0 ** -24
    x[8] = -0.0
    x[9, 0, 1:] = 0
    if dtype == inputs.BF16:
        x[10, 0, :32] = np.float32(3.38e38)
        x[10, 0, 0] = np.float32(-3.38e38)
        x[11] = 0
        x[11, 0, 1] = np.float32(1e-40)  # below the normal numbers
    bits = inputs.to_bits(x, dtype)
    if dtype == inputs.BF16:
        bits[11, 0, 1] = 0x0003
    cache = fa.int4_cache(1, 1, 16, 64)
    slots = np.arange(12, dtype=np.int32)
    fa.cache_append_int4(_t16(bits, dtype), _t16(bits, dtype), _dev(slots), *cache)
    zc, zw = np.zeros((1, 1, 16, 32), np.uint8), np.zeros((1, 1, 16, 2), np.int32)
    want_c, want_w = ref.append(inputs.bits_to_f64(bits, dtype), slots, zc, zw, 16, 32)
    for c, w in ((cache[0], cache[2]), (cache[1], cache[3])):
        assert np.array_equal(w.cpu().numpy(), want_w)
        assert np.array_equal(c.cpu().numpy(), want_c)
    # groups around a value that is no number are whole
    v = ref.values(want_c, want_w)[0, 0]
    assert np.isnan(v[3, :32]).all() and np.isfinite(v[3, 32:]).all() and np.isnan(v[4, 32:]).all()


@pytest.mark.parametrize("stride", ["odd", "repeated", "offset"])
def test_append_any_strides(stride):
    rng = np.random.default_rng(11)
    T, Hkv, d = 19, 2, 64
    flat = _t16(_rows(rng, (T * Hkv * (d + 1) + 9,), inputs.FP16), inputs.FP16)
    if stride == "odd":
        k = flat.as_strided((T, Hkv, d), (Hkv * (d + 1), d + 1, 1))
    elif stride == "repeated":
        k = flat[:d].expand(T, Hkv, d)
    else:
        k = flat[3:3 + T * Hkv * d].view(T, Hkv, d)
    v = k.flip(0)
    slots = rng.permutation(32)[:T].astype(np.int32)
    got, again = fa.int4_cache(2, Hkv, 16, d), fa.int4_cache(2, Hkv, 16, d)
    fa.cache_append_int4(k, v, _dev(slots), *got)
    fa.cache_append_int4(k.contiguous(), v, _dev(slots), *again)
    for a, b in zip(got, again):
        assert torch.equal(a, b)
    want, _ = ref.append(k.double().cpu().numpy(), slots, np.zeros((2, Hkv, 16, 32), np.uint8),
                         np.zeros((2, Hkv, 16, 2), np.int32), 16, 32)
    assert np.array_equal(got[0].cpu().numpy(), want)


@pytest.mark.parametrize("apart", [1, 2, 63, 64, 127])
def test_append_a_slot_named_twice_gets_the_later_row(apart):
    rng = np.random.default_rng(apart)
    T = 400
    slots = rng.permutation(511)[:T].astype(np.int32)
    slots[apart + 100] = slots[100]
    slots[apart + 3] = slots[3]
    slots[5], slots[5 + apart] = 511, 511
    slots[T - 1 - apart] = slots[T - 1]
    bits = _rows(rng, (T, 2, 128), inputs.BF16)
    seen = {}
    for t, s in enumerate(slots):  # no slot is named by rows farther apart
        assert s not in seen or t - seen[s] < 128
        seen[s] = t
        seen[s] = t
    cache = fa.int4_cache(32, 2, 16, 128)
    fa.cache_append_int4(_t16(bits, inputs.BF16), _t16(bits, inputs.BF16), _dev(slots), *cache)
    want_c, want_w = ref.append(inputs.bits_to_f64(bits, inputs.BF16), slots, np.zeros((32, 2, 16, 64), np.uint8),
                                np.zeros((32, 2, 16, 4), np.int32), 16, 32)
    assert np.array_equal(cache[0].cpu().numpy(), want_c) and np.array_equal(cache[3].cpu().numpy(), want_w)


# ------------------------------------------------------------- a problem's cache

def _problem(B, H, Hkv, Sq, d, group, bs, lens, dtype, seed=0, spread=1, far=0.0, junk=True, q_size=1.0):
    rng = np.random.default_rng(seed)
    lens = np.array(lens, np.int32)
    M = max(1, int(-(-lens.max() // bs)))
    need = [-(-int(n) // bs) for n in lens]
    pool = sum(need) + 3
    perm = rng.permutation(pool)
    table = np.full((B, M), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    codes = [rng.integers(0, 256, (pool, Hkv, bs, d // 2)).astype(np.uint8) for _ in range(2)]
    w = []
    for _ in range(2):
        s = 2.0 ** rng.integers(-spread, spread + 1, (pool, Hkv, bs, d // group)) * \
            (rng.integers(128, 256, (pool, Hkv, bs, d // group)) / 512.0)
        z = np.rint(7.5 + rng.standard_normal(s.shape) * 1.5 + far * rng.standard_normal(s.shape))
        w.append(ref.words(s.astype(np.float32), z))
    if junk:  # what no request sees: words that are no numbers
        for b, n in enumerate(lens):
            if n % bs:
                for x in w:
                    x[table[b, need[b] - 1], :, n % bs:] = rng.choice(
                        np.array([0x7FC07E00, 0x7F807C00, -1, 0x7F7F7BFF], np.int64), (Hkv, bs - n % bs, d // group))
        for block in perm[at:]:
            for x in w:
                x[block] = 0x7FC07E00
    qb = inputs.to_bits((rng.standard_normal((B, H, Sq, d)) * q_size).astype(np.float32), dtype)
    return dict(q=qb, kc=codes[0], vc=codes[1], kw=w[0], vw=w[1], table=table, lens=lens, bs=bs, dtype=dtype,
                group=group)


def _device(p):
    return [_t16(p["q"], p["dtype"])] + [_dev(p[n]) for n in ("kc", "vc", "kw", "vw", "table", "lens")]


# ------------------------------------------------------------------ reading back

@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
@pytest.mark.parametrize("layout", ["own", "inside", "odd", "tokens"])
@pytest.mark.parametrize("B,Hkv,d,group,bs,lens,rows,starts", [
    (1, 1, 64, 32, 16, [1], 1, None), (3, 2, 128, 32, 16, [40, 0, 17], 40, None),
    (2, 3, 256, 64, 64, [130, 700], 300, [100, -7]), (4, 1, 64, 64, 32, [5, 64, 33, 1], 200, [0, 64, -40, 3]),
    (2, 5, 128, 64, 128, [1000, 129], 513, [490, 2000])])
def test_read_back(B, Hkv, d, group, bs, lens, rows, starts, layout, dtype):
    p = _problem(B, Hkv, Hkv, 1, d, group, bs, lens, dtype, seed=B + d + rows, far=50.0)
    dt = DTYPES[dtype]
    shape = (B, Hkv, rows, d)
    if layout == "own":
        outs = [None, None]
    elif layout == "inside":
        outs = [torch.full((B, Hkv, rows + 9, d), 7.0, dtype=dt, device="cuda")[:, :, 4:4 + rows] for _ in range(2)]
    elif layout == "odd":
        outs = [torch.full((B * Hkv * rows * (d + 1),), 7.0, dtype=dt, device="cuda").as_strided(
            shape, (Hkv * rows * (d + 1), rows * (d + 1), d + 1, 1)) for _ in range(2)]
    else:  # K and V beside each other in a packed tensor, token by token
        both = torch.full((B, rows, 2 * Hkv, d), 7.0, dtype=dt, device="cuda")
        outs = [both[:, :, :Hkv].transpose(1, 2), both[:, :, Hkv:].transpose(1, 2)]
    st = None if starts is None else _dev(np.array(starts, np.int32))
    k, v = fa.cache_read_int4(*_device(p)[1:], rows, starts=st, dtype=dt, out_k=outs[0], out_v=outs[1])
    for got, c, w in ((k, p["kc"], p["kw"]), (v, p["vc"], p["vw"])):
        want = torch.full(shape, 0.0 if layout == "own" else 7.0, dtype=torch.float64)
        for b, L in enumerate(lens):
            x = ref.gathered(c, w, p["table"][b], L, bs)
            first = starts[b] if starts else 0
            for i in range(rows):
                if 0 <= first + i < L:
                    want[b, :, i] = torch.from_numpy(x[:, first + i])
        # s (c - z) has at most 8 + 12 bits, exact in fp32; then one rounding
        assert torch.equal(got.cpu(), want.float().to(dt))


@pytest.mark.parametrize("start", [-2 ** 31, -2 ** 31 + 1, 2 ** 31 - 1, -40, 39, 40])
def test_read_back_from_far_outside_a_request(start):
    p = _problem(2, 2, 2, 1, 64, 32, 16, [40, 40], inputs.BF16, seed=4)
    k, v = fa.cache_read_int4(*_device(p)[1:], 60, starts=_dev(np.array([start, 0], np.int32)))
    for got, c, w in ((k, p["kc"], p["kw"]), (v, p["vc"], p["vw"])):
        want = torch.zeros(2, 2, 60, 64, dtype=torch.float64)
        for b, first in enumerate((start, 0)):
            x = torch.from_numpy(ref.gathered(c, w, p["table"][b], 40, 16))
            for i in range(60):
                if 0 <= first + i < 40:
                    want[b, :, i] = x[:, first + i]
        assert torch.equal(got.cpu(), want.float().to(torch.bfloat16))


def test_read_back_entries_outside_the_pool_read_zeros():
    p = _problem(2, 1, 1, 1, 64, 32, 16, [40, 33], inputs.BF16, seed=3)
    p["table"][0, 1] = -1
    p["table"][1, 0] = len(p["kc"])
    k, v = fa.cache_read_int4(*_device(p)[1:], 40)
    for got, c, w in ((k, p["kc"], p["kw"]), (v, p["vc"], p["vw"])):
        for b, L in enumerate((40, 33)):
            want = torch.from_numpy(ref.gathered(c, w, p["table"][b], L, 16)).float().to(torch.bfloat16)
            assert torch.equal(got[b, :, :L].cpu(), want)


# ------------------------------------------------------------------ attention

def _check(p, o, lse, mask, max_len, scale=None):
    """Scores: a group's products are exact; their fp32 sums begin with the zeros' share and are cut off
    rather than rounded by at most 2^-23 of what they hold at each of up to 16 steps, and the groups are
    added in up to 9 roundings: 2^-18 of sum |q| s (15 + |z|).  Also the exponent's and the logarithm's few
    steps.  O: a weight times its scale is rounded to fp16, 2^-11 of it at most, and the zeros meet the
    rounded weight, so that is relative to p |v|; the sums of weights times codes and of weights times
    zeros, apart, lose at most 2^-17 of sum p s (15 + |z|) (cut off at 2^-23 of what they hold, a step per
    16 keys, the keys' signs alternating; 2^-23 per step over at most 64 steps of a warp in these lengths);
    below 2^-14 of the row's largest product a weight is off by a fixed 2^-25 of it, of up to 15 + |z|
    codes, which is inside 2^-17 of `big` unless scales are far apart.  O is rounded once."""
    d = p["q"].shape[-1]
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    q = inputs.bits_to_f64(p["q"], p["dtype"])
    want, want_lse, spread, reach, big = ref.decode(q, p["kc"], p["vc"], p["kw"], p["vw"], p["table"], p["lens"],
                                                    max_len, scale, mask, p["bs"])
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    none = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(lse), none) and np.all(o[none] == 0)
    tol = 2.0 ** -18 * reach + 2.0 ** -20 * (1 + np.abs(np.where(none, 0, want_lse)))
    err = np.abs(np.where(none, 0, lse) - np.where(none, 0, want_lse))
    assert np.all(err <= tol), float((err / tol).max())
    bound = (2.0 ** -11 + 2 * tol[..., None]) * spread + 2.0 ** -17 * big + U[p["dtype"]] * np.abs(want) + 2.0 ** -25
    err = np.abs(o - want)
    assert np.all(err <= bound), float((err / bound).max())
    return float((err / bound).max())


CASES = [
    # B, H, Hkv, Sq, d, group, bs, lens
    (1, 1, 1, 1, 64, 32, 16, [1]),
    (1, 1, 1, 1, 128, 64, 16, [16]),
    (3, 4, 4, 1, 128, 32, 16, [17, 1, 130]),
    (2, 8, 2, 1, 128, 32, 64, [128, 129]),
    (2, 5, 5, 2, 64, 64, 32, [127, 300]),
    (2, 6, 2, 3, 256, 32, 128, [255, 384]),
    (2, 32, 4, 1, 256, 64, 64, [700, 1]),
    (2, 16, 2, 5, 128, 64, 32, [333, 64]),
    (1, 128, 1, 1, 128, 32, 16, [500]),
    (1, 64, 1, 2, 64, 64, 128, [1000]),
    (1, 30, 1, 1, 64, 32, 16, [640]),
    (2, 7, 1, 9, 256, 32, 16, [77, 513]),
    (1, 24, 2, 1, 256, 32, 32, [600]),
    (2, 12, 1, 1, 64, 64, 16, [50, 1025]),
    (5, 3, 3, 1, 128, 32, 128, [0, 5, 0, 128, 4000]),
    (1, 2, 2, 1, 64, 32, 16, [9000]),
    (1, 8, 1, 4, 128, 64, 64, [6001]),
]


@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
@pytest.mark.parametrize("mask", ["causal", "none"])
@pytest.mark.parametrize("case", CASES)
def test_against_the_formula(case, mask, dtype):
    p = _problem(*case, dtype, seed=sum(case[:7]))
    max_len = max(1, int(p["lens"].max()))
    o, lse = fa.decode_paged_int4(*_device(p), max_len, mask=mask)
    _check(p, o, lse, mask, max_len)


@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (256, 32), (256, 64)])
def test_zeros_far_from_the_codes(d, group, dtype):
    p = _problem(2, 8, 2, 1, d, group, 16, [500, 77], dtype, seed=d + group, far=300.0, q_size=0.05)
    o, lse = fa.decode_paged_int4(*_device(p), 500)
    _check(p, o, lse, "none", 500)
