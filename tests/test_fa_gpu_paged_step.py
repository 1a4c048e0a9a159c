"""The paged cache's bookkeeping (fa_paged_update) and the quantising append
(fa_cache_append_fp8) on the GPU, against one-at-a-time implementations: whole
numbers and codes have to be equal."""
import numpy as np
import pytest

import step_reference as ref
from exact_io_aware_30_gb300 import fa, inputs

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from exact_io_aware_30_gb300 import build
    build.build()
    fa.load()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    assert fa.device_error() == fa.FA_OK


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


# ------------------------------------------------------------------ paged update

def _pool(rng, B, M, bs, spare=0, ring_size=None, lens=None):
    """A consistent cache: tables of the live blocks, the others in the ring from a random place on."""
    lens = rng.integers(0, M * bs + 1, B) if lens is None else np.array(lens)
    blocks = -(-lens // bs)
    pool = int(blocks.sum()) + spare
    ring_size = max(1, pool) if ring_size is None else ring_size
    perm = rng.permutation(max(1, pool))
    table = np.full((B, M), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :blocks[b]] = perm[at:at + blocks[b]]
        at += blocks[b]
    ring = np.full(ring_size, -7, np.int32)
    head = int(rng.integers(0, ring_size))
    ring[(head + np.arange(spare)) % ring_size] = perm[at:at + spare]
    return lens.astype(np.int32), table, ring, np.array([head, spare], np.int32)


def _compare(lens, delta, table, ring, state, bs, rows, in_place=False):
    want = ref.paged_update(lens, delta, table, ring, state, bs, rows)
    t, r, l, s = _i32(table), _i32(ring), _i32(lens), _i32(state)
    # rows past the end of the outputs stay as they are
    slot, pos = torch.full((rows + 5,), 77, dtype=torch.int32, device="cuda"), torch.full((rows + 5,), 78, dtype=torch.int32, device="cuda")
    kw = dict(seq_lens_out=l, ring_state_out=s) if in_place else {}
    got = fa.paged_update(l, _i32(delta), t, r, s, bs, slot_map=slot[:rows], positions=pos[:rows], **kw)
    for name in ("seq_lens", "status", "slot_map", "positions", "ring_state"):
        assert np.array_equal(getattr(got, name).cpu().numpy(), want[name]), name
    assert np.array_equal(t.cpu().numpy(), want["block_table"]) and np.array_equal(r.cpu().numpy(), want["free_ring"])
    assert bool((slot[rows:] == 77).all()) and bool((pos[rows:] == 78).all())
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("B,M,rows", [(1, 1, 1), (1, 3, 0), (2, 4, 7), (31, 5, 200), (64, 9, 64), (1024, 3, 2049),
                                      (1025, 4, 5000), (2500, 2, 20000)])
def test_update_against_one_request_after_another(B, M, rows, bs, in_place):
    rng = np.random.default_rng(B + bs)
    # few spare blocks: some requests run out; some deltas pass the table, the rows or the length
    lens, table, ring, state = _pool(rng, B, M, bs, spare=int(rng.integers(0, 2 * B + 1)))
    delta = rng.integers(-2 * bs, max(2, 2 * rows // B + 2), B)
    delta[rng.random(B) < 0.2] = 0
    delta[rng.random(B) < 0.1] = -(2 ** 31)
    delta[rng.random(B) < 0.02] = 2 ** 31 - 1
    _compare(lens, delta, table, ring, state, bs, rows, in_place)


def test_update_each_refusal_and_what_follows():
    rng = np.random.default_rng(1)
    # too long, no rows, no blocks, then one that needs no block, then one that needs one
    lens, table, ring, state = _pool(rng, 6, 4, 16, spare=2, lens=[60, 5, 16, 32, 3, 48])
    # (refused requests' rows count too: 10 + 40 + 33 + 17 = 100 are all there are)
    want = _compare(lens, [10, 40, 33, 17, 2, 1], table, ring, state, 16, 100)
    assert list(want["status"]) == [2, 0, 1, 1, 3, 3]
    want = _compare(lens, [10, 40, 33, 17, 2, 1], table, ring, state, 16, 200)
    assert list(want["status"]) == [2, 0, 1, 1, 0, 1]
    want = _compare(lens, [1, 40, 20, 0, 9, 1], table, ring, state, 16, 45)
    assert list(want["status"]) == [0, 0, 3, 0, 3, 3]


def test_update_lengths_outside_the_table_and_bad_state():
    rng = np.random.default_rng(2)
    lens, table, ring, state = _pool(rng, 4, 3, 16, spare=5, lens=[48, 0, 20, 7])
    _compare(np.array([1000, -5, 20, 7]), [-3, 4, 0, 12], table, ring, state, 16, 20)
    # a full ring drops what does not fit; a table entry below 0 gives slot -1
    ring_full = np.arange(6, dtype=np.int32)
    _compare(lens, [-48, 0, -20, 0], table, ring_full, np.array([3, 5]), 16, 4)
    table[3, 0] = -1
    want = _compare(lens, [0, 0, 0, 5], table, ring, state, 16, 9)
    assert list(want["slot_map"][:5]) == [-1] * 5
    # a block whose slots pass 31 bits
    table[3, 0] = 2 ** 27
    assert list(_compare(lens, [0, 0, 0, 1], table, ring, state, 16, 2)["slot_map"]) == [-1, -1]


def test_update_runs_as_a_replayed_graph():
    rng = np.random.default_rng(4)
    B, M, bs = 9, 12, 16
    lens, table, ring, state = _pool(rng, B, M, bs, spare=40, lens=rng.integers(0, 100, B))
    l, t, r, s = _i32(lens), _i32(table), _i32(ring), _i32(state)
    delta = _i32(np.ones(B))
    bufs = dict(slot_map=_i32(np.zeros(16)), positions=_i32(np.zeros(16)), status=_i32(np.zeros(B)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.paged_update(l, delta, t, r, s, bs, seq_lens_out=l, ring_state_out=s, **bufs)
    for step in range(40):
        change = rng.integers(-20, 3, B) if step % 5 == 4 else np.ones(B)
        delta.copy_(_i32(change))
        graph.replay()
        want = ref.paged_update(lens, change, table, ring, state, bs, 16)
        for name in ("seq_lens", "status", "slot_map", "positions", "ring_state"):
            assert np.array_equal(getattr(got, name).cpu().numpy(), want[name]), (step, name)
        lens, table, ring, state = (want[n] for n in ("seq_lens", "block_table", "free_ring", "ring_state"))
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), ring)
    # every block is in one place
    live = [int(x) for b in range(B) for x in table[b, :-(-int(lens[b]) // bs)]]
    free = [int(ring[(state[0] + i) % len(ring)]) for i in range(state[1])]
    assert len(set(live + free)) == len(live + free)


def test_update_refusals():
    l, t, r, s = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (2, 8, 4, 2))
    t = t.view(2, 4)
    ok = dict(max_tokens=4)
    fa.paged_update(l, l.clone(), t, r, s, 16, **ok)
    for bad in (lambda: fa.paged_update(l, l.clone(), t, r, s, 16), lambda: fa.paged_update(l, l.clone(), t, r, s, 17, **ok),
                lambda: fa.paged_update(l, l.clone().long(), t, r, s, 16, **ok),
                lambda: fa.paged_update(l, l[:1], t, r, s, 16, **ok), lambda: fa.paged_update(l, l.clone(), t.t(), r, s, 16, **ok),
                lambda: fa.paged_update(l, l.clone(), t, r, l, 16, seq_lens_out=t[0, :2], **ok),
                lambda: fa.paged_update(l, l.clone(), t, r, s, 16, seq_lens_out=s, ring_state_out=l, **ok),
                lambda: fa.paged_update(l, l.clone(), t, r, s, 16, slot_map=r, positions=r),
                lambda: fa.paged_update(l.cpu(), l, t, r, s, 16, **ok), lambda: fa.paged_update(l, l.cpu(), t, r, s, 16, **ok)):
        with pytest.raises(fa.FAError):
            bad()


# ------------------------------------------------------------------ append

def _rows(rng, T, Hkv, d, dtype):
    x = rng.standard_normal((T, Hkv, d)) * 2.0 ** rng.integers(-12, 8, (T, 1, 1))
    bits = inputs.to_bits(x.astype(np.float32), dtype)
    return bits, inputs.bits_to_f64(bits, dtype)


def _tensor16(bits, dtype):
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(
        torch.bfloat16 if dtype == inputs.BF16 else torch.float16)
    return t.cuda()


def _cache(rng, blocks, Hkv, bs, d, powers=True):
    codes = rng.integers(0, 256, (2, blocks, Hkv, bs, d)).astype(np.uint8)  # NaN codes among them
    scale = (2.0 ** rng.integers(-9, 3, (2, blocks, Hkv))).astype(np.float32)
    if not powers:
        scale *= rng.uniform(1, 2, scale.shape).astype(np.float32)
    return codes, scale


def _same_codes(a, b):
    """Equal, or both NaN (0x7F and 0xFF)."""
    return bool(np.all((a == b) | (((a & 0x7F) == 0x7F) & ((b & 0x7F) == 0x7F))))


def _check_append(kb, k, vb, v, slots, codes, scale, bs, dtype, views=None):
    t = [torch.from_numpy(c.copy()).cuda() for c in codes] + [torch.from_numpy(s.copy()).cuda() for s in scale]
    tk, tv = views if views else (_tensor16(kb, dtype), _tensor16(vb, dtype))
    fa.cache_append_fp8(tk, tv, _i32(slots), *t)
    for i, x in enumerate((k, v)):
        want_codes, want_scale = ref.append(x, slots, codes[i], scale[i], bs)
        assert np.array_equal(t[2 + i].cpu().numpy(), want_scale), np.argwhere(t[2 + i].cpu().numpy() != want_scale)[:4]
        assert _same_codes(t[i].cpu().numpy(), want_codes)
    return t


@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
@pytest.mark.parametrize("d,bs,Hkv", [(64, 16, 1), (64, 128, 3), (128, 16, 5), (128, 64, 2), (256, 32, 2), (256, 128, 1)])
@pytest.mark.parametrize("powers", [True, False])
def test_append_ragged_requests(d, bs, Hkv, dtype, powers):
    rng = np.random.default_rng(d + bs + Hkv)
    runs = [1, 1, 3, bs, bs - 1, bs + 1, 2 * bs + 5, 2, 1]
    blocks = sum(-(-n // bs) + 1 for n in runs) + 2
    perm, slots, at = rng.permutation(blocks), [], 0
    for n in runs:
        begin = int(rng.integers(0, bs))
        pos = begin + np.arange(n)
        slots += list(perm[at + pos // bs] * bs + pos % bs)
        at += -(-n // bs) + 1
    slots = np.array(slots)
    slots[rng.random(len(slots)) < 0.1] = -1
    kb, k = _rows(rng, len(slots), Hkv, d, dtype)
    vb, v = _rows(rng, len(slots), Hkv, d, dtype)
    codes, scale = _cache(rng, blocks, Hkv, bs, d, powers)
    _check_append(kb, k, vb, v, slots, codes, scale, bs, dtype)


def test_append_many_rows_share_ctas():
    # enough rows that a CTA takes several: leaders found behind earlier CTAs' rows, padding at the end
    rng = np.random.default_rng(11)
    bs, Hkv, d, T = 16, 4, 64, 6000
    blocks = 420
    pos = 5 + np.arange(T)
    slots = rng.permutation(blocks)[pos // bs] * bs + pos % bs
    slots[1000:1300] = -1
    slots[5500:] = -1
    kb, k = _rows(rng, T, Hkv, d, inputs.BF16)
    codes, scale = _cache(rng, blocks, Hkv, bs, d)
    _check_append(kb, k, kb, k, slots, codes, scale, bs, inputs.BF16)


def test_append_infinities_nan_zeros_and_tiny_values():
    rng = np.random.default_rng(12)
    for dtype in (inputs.BF16, inputs.FP16):
        kb, _ = _rows(rng, 8, 2, 64, dtype)
        inf, nan = (0x7F80, 0x7FC0) if dtype == inputs.BF16 else (0x7C00, 0x7E00)
        kb[0, 0, 3], kb[0, 0, 4], kb[0, 1, 5] = inf, inf | 0x8000, nan
        kb[1] = 0              # all zeros: the smallest scale
        kb[2, 0] = 1           # the type's smallest value
        kb[3] = inf            # nothing finite
        kb[4, 0], kb[5, 1] = nan, 0x7BFF
        k = inputs.bits_to_f64(kb, dtype)
        slots = np.array([0, 16, 32, 48, 65, 81, 97, 113])
        codes, scale = _cache(rng, 9, 2, 16, 64)
        scale[:, 4], scale[:, 5], scale[0, 6], scale[1, 6] = np.nan, np.inf, 0.0, -1.0
        t = _check_append(kb, k, kb, k, slots, codes, scale, 16, dtype)
        assert float(t[2][1].max()) == 2.0 ** -126


def test_append_border_values_of_the_scale():
    # amax exactly 448 s stays, one step above doubles the scale
    x = np.zeros((4, 1, 64), np.float32)
    x[0, 0, 0], x[1, 0, 0], x[2, 0, 0], x[3, 0, 0] = 448.0, 450.0, 1.75, -1.7578125
    bits = inputs.to_bits(x, inputs.BF16)
    k = inputs.bits_to_f64(bits, inputs.BF16)
    codes, scale = _cache(np.random.default_rng(0), 4, 1, 16, 64)
    t = _check_append(bits, k, bits, k, np.arange(4) * 16, codes, scale, 16, inputs.BF16)
    assert t[2][:, 0].tolist() == [1.0, 2.0, 2.0 ** -8, 2.0 ** -7]


def test_append_a_slot_named_twice_gets_the_later_row():
    rng = np.random.default_rng(13)
    kb, k = _rows(rng, 6, 2, 128, inputs.FP16)
    codes, scale = _cache(rng, 3, 2, 32, 128)
    _check_append(kb, k, kb, k, np.array([40, 33, 40, 50, 33, 34]), codes, scale, 32, inputs.FP16)


def test_append_slots_outside_the_pool_are_skipped():
    rng = np.random.default_rng(14)
    kb, k = _rows(rng, 7, 2, 64, inputs.BF16)
    codes, scale = _cache(rng, 3, 2, 16, 64)
    _check_append(kb, k, kb, k, np.array([-1, 48, 47, -2 ** 31, 2 ** 31 - 1, 3, 49]), codes, scale, 16, inputs.BF16)
    _check_append(kb, k, kb, k, np.full(7, -1), codes, scale, 16, inputs.BF16)


def test_append_token_by_token_equals_the_reference():
    rng = np.random.default_rng(15)
    kb, k = _rows(rng, 40, 2, 64, inputs.BF16)
    codes, scale = _cache(rng, 4, 2, 16, 64)
    t = [torch.from_numpy(c.copy()).cuda() for c in codes] + [torch.from_numpy(s.copy()).cuda() for s in scale]
    want = [(codes[0], scale[0]), (codes[1], scale[1])]
    x = _tensor16(kb, inputs.BF16)
    for i in range(40):
        slot = np.array([7 + i])
        fa.cache_append_fp8(x[i:i + 1], x[i:i + 1], _i32(slot), *t)
        want = [ref.append(k[i:i + 1], slot, c, s, 16) for c, s in want]
    for i in range(2):
        assert _same_codes(t[i].cpu().numpy(), want[i][0]) and np.array_equal(t[2 + i].cpu().numpy(), want[i][1])


def test_append_strided_and_unaligned_rows_and_fp8_typed_caches():
    rng = np.random.default_rng(16)
    T, Hkv, d, bs = 37, 3, 64, 32
    bits, x = _rows(rng, T, 2 * Hkv, d + 2, inputs.BF16)
    packed = _tensor16(bits, inputs.BF16)
    slots = 5 + np.arange(T)
    codes, scale = _cache(rng, 3, Hkv, bs, d)
    for lo in (0, 1):
        views = packed[:, :Hkv, lo:lo + d], packed[:, Hkv:, lo:lo + d]
        _check_append(None, x[:, :Hkv, lo:lo + d], None, x[:, Hkv:, lo:lo + d], slots, codes, scale, bs, inputs.BF16, views)
    # [B, Hkv, S, d] as rope writes it, seen as tokens; one row for every head (stride 0)
    bits, x = _rows(rng, Hkv, T, d, inputs.FP16)
    view = _tensor16(bits, inputs.FP16).transpose(0, 1)
    one = view[:, :1].expand(T, Hkv, d)
    _check_append(None, x.transpose(1, 0, 2), None, np.repeat(x.transpose(1, 0, 2)[:, :1], Hkv, 1), slots, codes, scale,
                  bs, inputs.FP16, (view, one))
    t = [torch.from_numpy(c.copy()).cuda().view(torch.float8_e4m3fn) for c in codes] + \
        [torch.from_numpy(s.copy()).cuda() for s in scale]
    fa.cache_append_fp8(view, one, _i32(slots), *t)
    want, _ = ref.append(x.transpose(1, 0, 2), slots, codes[0], scale[0], bs)
    assert _same_codes(t[0].view(torch.uint8).cpu().numpy(), want)


def test_append_empty_and_refusals():
    rng = np.random.default_rng(17)
    codes, scale = _cache(rng, 3, 2, 16, 64)
    t = [torch.from_numpy(c.copy()).cuda() for c in codes] + [torch.from_numpy(s.copy()).cuda() for s in scale]
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    s = _i32([0, 1, 2, 3])
    fa.cache_append_fp8(x[:0], x[:0], s[:0], *t)
    assert np.array_equal(t[0].cpu().numpy(), codes[0])
    for bad in (lambda: fa.cache_append_fp8(x.float(), x.float(), s, *t), lambda: fa.cache_append_fp8(x, x.half(), s, *t),
                lambda: fa.cache_append_fp8(x, x, s.long(), *t), lambda: fa.cache_append_fp8(x, x, s[:3], *t),
                lambda: fa.cache_append_fp8(x[:, :1], x[:, :1], s, *t), lambda: fa.cache_append_fp8(x, x, s, t[0], t[0], t[2], t[3]),
                lambda: fa.cache_append_fp8(x, x, s, t[0], t[1], t[2], t[2]),
                lambda: fa.cache_append_fp8(x, x, s, t[0].float(), t[1], t[2], t[3]),
                lambda: fa.cache_append_fp8(x.cpu(), x, s, *t), lambda: fa.cache_append_fp8(x, x, s, t[0].cpu(), t[1], t[2], t[3]),
                lambda: fa.cache_append_fp8(x[..., ::2], x[..., ::2], s, *t)):
        with pytest.raises(fa.FAError):
            bad()


def test_append_past_32_bit_offsets():
    # a pool of over 2^32 bytes: its last blocks are written, nothing else changes
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    bs, Hkv, d = 128, 8, 256
    blocks = (1 << 32) // (bs * Hkv * d) + 3
    kc = torch.zeros(blocks, Hkv, bs, d, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    ks, vs = torch.ones(blocks, Hkv, device="cuda"), torch.ones(blocks, Hkv, device="cuda")
    x = torch.full((3, Hkv, d), 448.0, dtype=torch.bfloat16, device="cuda")
    fa.cache_append_fp8(x, x, _i32([(blocks - 1) * bs + 5, (blocks - 2) * bs, 7]), kc, vc, ks, vs)
    for c in (kc, vc):
        assert bool((c[-1, :, 5] == 0x7E).all()) and bool((c[-2, :, 0] == 0x7E).all()) and bool((c[0, :, 7] == 0x7E).all())
        assert int((c[-4:].int() != 0).sum()) == 2 * Hkv * d and int((c[:4].int() != 0).sum()) == Hkv * d
