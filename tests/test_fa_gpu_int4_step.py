"""Attention over the 4-bit paged cache where it can go wrong -- scales far apart,
values that are no numbers, masks that leave rows empty, streams, graphs, threads --
and the decode step as a program uses it: bookkeeping, rotary positions, append,
reading back and attention in a row."""
import threading

import numpy as np
import pytest

import int4_reference as ref
import test_fa_gpu_int4 as base
from exact_io_aware_30_gb300 import fa, inputs

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

_problem, _device, _check, _dev = base._problem, base._device, base._check, base._dev


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from exact_io_aware_30_gb300 import build
    build.build()
    fa.load()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    assert fa.device_error() == fa.FA_OK


def _scales(p, name, s):
    """Replaces a cache's scales (powers of two here), zeros kept."""
    _, z = ref.unpack_words(p[name])
    z = np.where(np.isfinite(z), z, 0.0)
    p[name] = ref.words(np.broadcast_to(s, z.shape).astype(np.float32), z)


def _check_far(p, o, lse, max_len):
    """As _check, with V scales far apart.  A row's reference is at most 2^14 above its largest product of a
    weight and a scale over its group's reference (6 that it keeps ahead, 8 that a scale may lie above the
    reference), of which 2^12 is room: fp16's smallest half step 2^-25 is at most 2^-23 of that product.  A
    group's own products may lie up to 2^8 lower (its scales within 2^8 of the reference): 2^-15 of its
    largest product, for each key whose product is that far down.  Those lie below 2^-14 of it and 2^10 times
    their rounding; with n keys n 2^-23 of the largest, and 2^-15 for those near it."""
    d = p["q"].shape[-1]
    q = inputs.bits_to_f64(p["q"], p["dtype"])
    want, want_lse, spread, reach, big = ref.decode(q, p["kc"], p["vc"], p["kw"], p["vw"], p["table"], p["lens"],
                                                    max_len, 1 / np.sqrt(d), "none", p["bs"])
    err = np.abs(lse.double().cpu().numpy() - want_lse)
    tol = 2.0 ** -18 * reach + 2.0 ** -20 * (1 + np.abs(want_lse))
    assert np.all(err <= tol)
    n = max_len
    bound = (2.0 ** -11 + 2 * tol[..., None]) * spread + (2.0 ** -15 + n * 2.0 ** -23) * big + \
        base.U[p["dtype"]] * np.abs(want) + 2.0 ** -25
    got = o.double().cpu().numpy()
    most = 65504.0 if p["dtype"] == inputs.FP16 else 3.3895e38
    over = np.isinf(got) & (np.sign(got) == np.sign(want)) & (np.abs(want) + bound > most)  # past the type's largest
    err = np.abs(np.where(over, want, got) - want)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
@pytest.mark.parametrize("H,Hkv,d,group", [(4, 4, 64, 64), (8, 2, 128, 32), (16, 2, 128, 64), (3, 1, 256, 32), (24, 1, 64, 32)])
@pytest.mark.parametrize("kind", ["tokens", "groups", "falling", "rising", "zeros", "tiny", "huge"])
def test_v_scales_far_apart(H, Hkv, d, group, kind, dtype):
    p = _problem(2, H, Hkv, 1, d, group, 16, [400, 61], dtype, seed=H + d, junk=False)
    rng = np.random.default_rng(3)
    shape = p["vw"].shape
    if kind == "tokens":  # any token may outweigh all others
        s = 2.0 ** rng.integers(-20, 21, (*shape[:3], 1))
    elif kind == "groups":
        s = 2.0 ** rng.integers(-20, 21, (1, 1, 1, shape[3]))
    elif kind in ("falling", "rising"):  # request 0's first tokens set references that its later ones leave far behind
        s = np.ones(shape[:3] + (1,))
        sign = -1.0 if kind == "falling" else 1.0
        for i, block in enumerate(p["table"][0]):
            s[block] = 2.0 ** (sign * 2 * i)
    elif kind == "zeros":
        s = np.where(rng.random((*shape[:3], 1)) < 0.5, 0.0, 1.0) * np.ones(shape)
        s[p["table"][1]] = 0.0
    else:
        s = np.float64(2.0 ** (-120 if kind == "tiny" else 100))
    _scales(p, "vw", s)
    o, lse = fa.decode_paged_int4(*_device(p), 400)
    if kind == "huge" and dtype == inputs.FP16:  # past the type
        assert bool(torch.isinf(o).any()) and not bool(torch.isnan(o).any())
        return
    _check_far(p, o, lse, 400)


def test_a_heavy_key_with_a_tiny_scale_does_not_hide_light_keys_with_large_ones():
    # key 3 carries all but 2^-20 of the weight, with values 2^-30; the others' products outweigh it
    n, d = 600, 128
    p = _problem(1, 2, 1, 1, d, 32, 16, [n], inputs.BF16, seed=9, junk=False)
    _scales(p, "kw", 0.0)
    s = np.ones(p["vw"].shape)
    first = p["table"][0, 0]
    s[first, 0, 3] = 2.0 ** -30
    _scales(p, "vw", s)
    q = np.zeros((1, 2, 1, d))
    q[..., 0] = 1.0
    p["q"] = inputs.to_bits(q.astype(np.float32), inputs.BF16)
    p["kw"][first, 0, 3] = ref.words(np.array([1.0] * 4, np.float32), np.array([1.0] * 4))
    p["kc"][first, 0, 3] = 0x11
    p["kc"][first, 0, 3, 0] = 0x1F  # 15 - 1 = 14 nats above the others
    o, lse = fa.decode_paged_int4(*_device(p), n, scale=1.0)
    _check(p, o, lse, "none", n, 1.0)


@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
def test_score_scale_zero_small_and_large(dtype):
    p = _problem(2, 8, 2, 1, 128, 32, 16, [300, 45], dtype, seed=40)
    for scale in (0.0, 1e-30, 1.0):
        o, lse = fa.decode_paged_int4(*_device(p), 300, scale=scale)
        _check(p, o, lse, "none", 300, scale)


@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
@pytest.mark.parametrize("size", [1e-4, 30.0])
def test_query_rows_of_very_different_sizes(dtype, size):
    p = _problem(1, 8, 1, 2, 128, 64, 16, [300], dtype, seed=41, q_size=size)
    q = inputs.bits_to_f64(p["q"], dtype)
    q[:, 0] = 0.0
    q[:, 1, :, 1:] = 0.0
    q[:, 2] *= 2.0 ** -6
    q[:, 3, :, 5] = 8.0  # one large component beside small ones
    p["q"] = inputs.to_bits(q.astype(np.float32), dtype)
    o, lse = fa.decode_paged_int4(*_device(p), 300)
    _check(p, o, lse, "none", 300)


def test_rows_in_front_of_the_first_token_see_nothing():
    p = _problem(3, 4, 2, 4, 128, 32, 16, [2, 0, 5], inputs.BF16, seed=43)
    o, lse = fa.decode_paged_int4(*_device(p), 5, mask="causal")
    _check(p, o, lse, "causal", 5)
    assert bool((o[0, :, :2] == 0).all()) and bool(torch.isneginf(lse[1]).all())


def test_lengths_outside_the_bound_are_clamped():
    p = _problem(3, 4, 2, 1, 64, 32, 16, [48, 48, 3], inputs.BF16, seed=44)
    dev = _device(p)
    dev[6] = torch.tensor([1000, -5, 3], dtype=torch.int32, device="cuda")
    o, lse = fa.decode_paged_int4(*dev, 48)
    p["lens"] = np.array([48, 0, 3], np.int32)
    _check(p, o, lse, "none", 48)


@pytest.mark.parametrize("d,group,bs", [(128, 32, 16), (64, 64, 32), (256, 64, 128)])
def test_blocks_outside_the_pool_read_zeros(d, group, bs):
    p = _problem(2, 8, 2, 1, d, group, bs, [6 * bs + 4, 4 * bs], inputs.BF16, seed=45)
    p["table"][0, 1], p["table"][0, 4], p["table"][1, 0] = -1, 10 ** 6, -2 ** 31
    o, lse = fa.decode_paged_int4(*_device(p), 6 * bs + 4)
    _check(p, o, lse, "none", 6 * bs + 4)


def test_queries_that_are_no_numbers_give_nan_in_their_own_rows_only():
    for dtype, inf, nan in ((inputs.BF16, 0x7F80, 0x7FC0), (inputs.FP16, 0x7C00, 0x7E00)):
        for H in (8, 12):  # four and six rows to a K/V head
            p = _problem(1, H, 2, 1, 128, 32, 16, [700], dtype, seed=46)
            clean, clean_lse = fa.decode_paged_int4(*_device(p), 700)
            p["q"][0, 1, 0, 7], p["q"][0, 7, 0, 0] = inf, nan
            o, lse = fa.decode_paged_int4(*_device(p), 700)
            for h in range(H):
                if h in (1, 7):
                    assert bool(torch.isnan(o[0, h]).all()) and bool(torch.isnan(lse[0, h]).all())
                else:
                    assert torch.equal(o[0, h], clean[0, h]) and torch.equal(lse[0, h], clean_lse[0, h])


def test_query_rows_too_large_for_the_products_are_nan():
    p = _problem(1, 4, 2, 1, 64, 32, 16, [50], inputs.BF16, seed=47)
    _scales(p, "kw", 2.0 ** -105)  # (scores stay below 2^25)
    q = inputs.bits_to_f64(p["q"], inputs.BF16)
    q[0, 0, 0, 3], q[0, 3, 0, 3] = 2.0 ** 112, 2.0 ** 111
    p["q"] = inputs.to_bits(q.astype(np.float32), inputs.BF16)
    o, lse = fa.decode_paged_int4(*_device(p), 50)
    assert bool(torch.isnan(o[0, 0]).all()) and bool(torch.isnan(lse[0, 0]).all())
    assert bool(torch.isfinite(o[0, 1:]).all()) and bool(torch.isfinite(lse[0, 1:]).all())


def test_groups_that_are_no_numbers_stay_in_their_head_and_columns():
    p = _problem(2, 8, 2, 1, 128, 32, 16, [300, 40], inputs.BF16, seed=48)
    clean, clean_lse = fa.decode_paged_int4(*_device(p), 300)
    nan = np.int32(0x7FC00000)
    p["vw"][p["table"][0, 5], 1, 7, 2] = nan     # request 0, K/V head 1, components 64 .. 95
    p["kw"][p["table"][1, 1], 0, 3, 0] = nan     # request 1, K/V head 0: its scores
    o, lse = fa.decode_paged_int4(*_device(p), 300)
    assert bool(torch.isnan(o[0, 4:, :, 64:96]).all()) and bool(torch.isnan(o[1, :4]).all())
    assert bool(torch.isnan(lse[1, :4]).all())
    assert torch.equal(o[0, :4], clean[0, :4]) and torch.equal(o[1, 4:], clean[1, 4:])
    assert torch.equal(o[0, 4:, :, :64], clean[0, 4:, :, :64]) and torch.equal(o[0, 4:, :, 96:], clean[0, 4:, :, 96:])
    assert torch.equal(lse[0], clean_lse[0])


def test_two_calls_give_the_same_bits_and_outputs_can_be_given():
    p = _problem(4, 16, 4, 1, 128, 64, 16, [900, 33, 1, 2000], inputs.FP16, seed=47)
    dev = _device(p)
    a = fa.decode_paged_int4(*dev, 2000)
    out, lse = torch.empty_like(a[0]), torch.empty_like(a[1])
    st, n = fa.decode_int4_workspace_query(4, 16, 4, 1, 128, 64, 16, p["table"].shape[1], p["kc"].shape[0], 2000,
                                           dtype=fa.DTYPE_FP16)
    assert st == fa.FA_OK
    ws = torch.full((n + 256,), 0xAB, dtype=torch.uint8, device="cuda")  # its contents do not matter
    b = fa.decode_paged_int4(*dev, 2000, out=out, lse=lse, workspace=ws)
    assert b[0] is out and torch.equal(a[0], out) and torch.equal(a[1], lse)
    with pytest.raises(fa.FAError):
        fa.decode_paged_int4(*dev, 2000, workspace=ws[:n - 1])


@pytest.mark.parametrize("longest", [500, 900])  # units whole, units cut
@pytest.mark.parametrize("H,Hkv,Sq,d,group,dtype", [(24, 24, 1, 128, 32, inputs.FP16), (24, 24, 1, 128, 64, inputs.BF16),
                                                    (48, 24, 4, 64, 32, inputs.BF16), (24, 12, 8, 128, 32, inputs.FP16),
                                                    (24, 24, 2, 256, 32, inputs.BF16), (12, 12, 16, 256, 64, inputs.FP16)])
def test_many_short_units_give_the_same_bits_each_time(H, Hkv, Sq, d, group, dtype, longest):
    """A CTA's warps hand their sums to each other at each unit's end, thousands of times per call: what one
    hands on must not lie where another still reads.  Each of many calls gives the first's bits, and those are right."""
    lens = [longest - 13 * i for i in range(32)]
    p = _problem(len(lens), H, Hkv, Sq, d, group, 16, lens, dtype, seed=H + d + Sq)
    dev = _device(p)
    o, lse = fa.decode_paged_int4(*dev, longest)
    _check(p, o, lse, "none", longest)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        again, again_lse = fa.decode_paged_int4(*dev, longest)
        wrong += (again.view(torch.int16) != o.view(torch.int16)).sum() + (again_lse != lse).sum()
    assert int(wrong) == 0


def test_two_streams_at_once_and_two_graphs():
    ps = [_problem(4, 8, 2, 1, 128, 32, 16, [900 + i, 33, 1, 2000], inputs.BF16, seed=48 + i) for i in range(2)]
    devs = [_device(p) for p in ps]
    want = [fa.decode_paged_int4(*d, 2000) for d in devs]
    streams = [torch.cuda.Stream() for _ in devs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [fa.decode_paged_int4(*d, 2000, stream=s) for d, s in zip(devs, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    graphs, outs = [], []
    for d in devs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(fa.decode_paged_int4(*d, 2000))
        graphs.append(graph)
    for o, _ in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for g, w in zip(outs, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_refusals():
    p = _problem(2, 8, 2, 1, 128, 32, 16, [50, 20], inputs.BF16, seed=49)
    d = _device(p)
    fa.decode_paged_int4(*d, 50)

    def with_(i, x):
        return d[:i] + [x] + d[i + 1:]

    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.empty(2, 2, 9, 128, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: fa.decode_paged_int4(*with_(0, d[0].float()), 50), lambda: fa.decode_paged_int4(*with_(0, d[0][:, :7]), 50),
                lambda: fa.decode_paged_int4(*with_(1, d[1].float()), 50), lambda: fa.decode_paged_int4(*with_(1, d[1][..., :32]), 50),
                lambda: fa.decode_paged_int4(*with_(3, d[3].float()), 50), lambda: fa.decode_paged_int4(*with_(4, d[4][..., :2]), 50),
                lambda: fa.decode_paged_int4(*with_(3, d[3][..., :3].contiguous()), 50),
                lambda: fa.decode_paged_int4(*with_(5, d[5].long()), 50), lambda: fa.decode_paged_int4(*with_(6, d[6][:1]), 50),
                lambda: fa.decode_paged_int4(*with_(6, d[6].cpu()), 50), lambda: fa.decode_paged_int4(*d, 0),
                lambda: fa.decode_paged_int4(*d, 65), lambda: fa.decode_paged_int4(*d, 50, mask="window"),
                lambda: fa.decode_paged_int4(*d, 50, out=d[0]), lambda: fa.decode_paged_int4(*d, 50, scale=float("inf")),
                lambda: fa.decode_paged_int4(*d, 50, lse=torch.empty(2, 8, 1, device="cuda").half()),
                lambda: fa.decode_paged_int4(*d, 50, workspace=ws[1:]),
                lambda: fa.cache_append_int4(k.cpu(), k, slots, *d[1:5]), lambda: fa.cache_append_int4(k, k[:2], slots, *d[1:5]),
                lambda: fa.cache_append_int4(k, k.half(), slots, *d[1:5]), lambda: fa.cache_append_int4(k, k, slots.long(), *d[1:5]),
                lambda: fa.cache_append_int4(k[:, :1], k[:, :1], slots, *d[1:5]),
                lambda: fa.cache_append_int4(k.transpose(0, 2), k.transpose(0, 2), slots, *d[1:5]),
                lambda: fa.cache_append_int4(k.float(), k.float(), slots, *d[1:5]),
                lambda: fa.cache_read_int4(*d[1:7], -1), lambda: fa.cache_read_int4(*d[1:7], 9, out_k=out),
                lambda: fa.cache_read_int4(*d[1:7], 9, out_k=out, out_v=out),
                lambda: fa.cache_read_int4(*d[1:7], 8, out_k=out, out_v=out.clone()),
                lambda: fa.cache_read_int4(*d[1:7], 9, dtype=torch.float16, out_k=out, out_v=out.clone()),
                lambda: fa.cache_read_int4(*d[1:7], 9, dtype=torch.float32),
                lambda: fa.cache_read_int4(*d[1:7], 9, starts=d[6][:1]),
                lambda: fa.cache_read_int4(*d[1:7], 9, out_k=out[:, :, :1].expand(2, 2, 9, 128), out_v=out.clone())):
        with pytest.raises(fa.FAError):
            bad()


def test_offsets_past_32_bits():
    if torch.cuda.mem_get_info()[0] < 32 << 30:
        pytest.skip("needs 32 GB")
    bs, Hkv, d, group, n = 128, 8, 256, 32, 300
    blocks = (1 << 32) // (bs * Hkv * d // 2) + 4
    p = _problem(1, 8, Hkv, 1, d, group, bs, [n], inputs.BF16, seed=50, junk=False)
    dev = _device(p)
    want, want_read = fa.decode_paged_int4(*dev, n), fa.cache_read_int4(*dev[1:7], n)
    kc, vc = (torch.full((blocks, Hkv, bs, d // 2), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((blocks, Hkv, bs, d // group), 0x7FC07E00, dtype=torch.int32, device="cuda") for _ in range(2))
    table = dev[5].clone()
    for i, at in enumerate((blocks - 1, 0, blocks - 2)):
        old = int(dev[5][0, i])
        kc[at], vc[at], ks[at], vs[at] = dev[1][old], dev[2][old], dev[3][old], dev[4][old]
        table[0, i] = at
    got = fa.decode_paged_int4(dev[0], kc, vc, ks, vs, table, dev[6], n)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for a, b in zip(fa.cache_read_int4(kc, vc, ks, vs, table, dev[6], n), want_read):
        assert torch.equal(a, b)
    # rows into the last block; its neighbours stay
    x = torch.randn(2, Hkv, d, device="cuda").bfloat16()
    before = [t[-2:].clone() for t in (kc, vc, ks, vs)]
    fa.cache_append_int4(x, x, torch.tensor([(blocks - 1) * bs + 7, (blocks - 2) * bs + 1], dtype=torch.int32, device="cuda"),
                         kc, vc, ks, vs)
    codes, words = ref.append(x.double().cpu().numpy(), np.array([bs + 7, 1]), before[0].cpu().numpy(),
                              before[2].cpu().numpy(), bs, group)
    for c, w in ((kc, ks), (vc, vs)):
        w2, w0 = (words, before[2]) if w is ks else (ref.append(x.double().cpu().numpy(), np.array([bs + 7, 1]),
                                                                before[1].cpu().numpy(), before[3].cpu().numpy(), bs, group)[1],
                                                     before[3])
        assert np.array_equal(w[-2:].cpu().numpy(), w2)
    assert np.array_equal(kc[-2:].cpu().numpy(), codes)


@pytest.mark.parametrize("H,Hkv,Sq,d", [(4, 4, 1, 64), (8, 1, 1, 128), (32, 1, 1, 128), (20, 1, 1, 256)])
def test_a_wait_that_runs_out_is_reported_and_the_context_recovers(H, Hkv, Sq, d):
    # one, eight, thirty-two and twenty rows per K/V head
    p = _problem(3, H, Hkv, Sq, d, 32, 16, [700, 3, 129], inputs.BF16, seed=51)
    dev = _device(p)
    assert fa.device_error() == fa.FA_OK
    fa.set_debug_stall_ms(50)
    try:
        fa.decode_paged_int4(*dev, 700, mask="causal")
        torch.cuda.synchronize()
    finally:
        fa.set_debug_stall_ms(0)
    assert fa.device_error() == fa.FA_ERR_DEVICE_TIMEOUT
    assert fa.device_error() == fa.FA_OK
    o, lse = fa.decode_paged_int4(*dev, 700, mask="causal")
    _check(p, o, lse, "causal", 700)


@pytest.mark.parametrize("B", [129, 700])
def test_more_requests_than_threads_with_uneven_lengths(B):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 200, B)
    lens[rng.integers(0, B)] = 2500
    p = _problem(B, 2, 1, 1, 64, 32, 16, lens, inputs.BF16, seed=52)
    o, lse = fa.decode_paged_int4(*_device(p), 2500)
    _check(p, o, lse, "none", 2500)


def test_a_unit_cut_into_many_pieces():
    # one request of one K/V head over the whole grid: more than 32 partials to merge
    p = _problem(1, 4, 1, 1, 64, 64, 128, [60000], inputs.BF16, seed=58)
    o, lse = fa.decode_paged_int4(*_device(p), 60000)
    _check(p, o, lse, "none", 60000)


def test_a_bound_far_above_the_lengths_and_a_wide_table():
    # the grid is sized by the bound; most of its CTAs find no tile
    p = _problem(3, 8, 2, 2, 128, 32, 16, [5, 300, 0], inputs.BF16, seed=53)
    wide = np.full((3, 9000), -1, np.int32)
    wide[:, :p["table"].shape[1]] = p["table"]
    p["table"] = wide
    narrow = fa.decode_paged_int4(*_device(p), 300, mask="causal")
    o, lse = fa.decode_paged_int4(*_device(p), 9000 * 16, mask="causal")
    _check(p, o, lse, "causal", 9000 * 16)
    _check(p, *narrow, "causal", 300)


def test_two_host_threads_at_once():
    ps = [_problem(3, 8, 2, 1, d, 32, 16, [700, 33, 1200], inputs.FP16, seed=54 + d) for d in (64, 128)]
    devs = [_device(p) for p in ps]
    want = [fa.decode_paged_int4(*d, 1200) + fa.cache_read_int4(*d[1:7], 1200) for d in devs]
    torch.cuda.synchronize()
    got, failed = [None, None], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(30):
                got[i] = fa.decode_paged_int4(*devs[i], 1200, stream=stream) + \
                    fa.cache_read_int4(*devs[i][1:7], 1200, stream=stream)
            stream.synchronize()
        except Exception as e:  # (an assertion in a thread would be lost)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a, b)


def test_the_results_of_the_kernel_in_front_are_seen():
    # the kernels begin before the one in front of them ends: each must still wait for its results
    p = _problem(2, 8, 2, 1, 128, 32, 16, [3000, 1500], inputs.BF16, seed=55)
    dev = _device(p)
    want, want_read = fa.decode_paged_int4(*dev, 3000), fa.cache_read_int4(*dev[1:7], 3000)
    plan, x = fa.rope_plan(128), torch.randn(1, 64, 8192, 128, device="cuda").bfloat16()
    big, q, lens = torch.empty_like(x), torch.zeros_like(dev[0]), torch.zeros_like(dev[6])
    rows = torch.randn(64, 2, 128, device="cuda").bfloat16()
    slots = torch.arange(64, dtype=torch.int32, device="cuda") + int(dev[5][1, 2]) * 16
    slots = torch.where(slots < (int(dev[5][1, 2]) + 1) * 16, slots, torch.full_like(slots, -1))
    fresh = [t.clone() for t in dev[1:5]]
    fa.cache_append_int4(rows, rows, slots, *dev[1:5])
    after, after_read = fa.decode_paged_int4(*dev, 3000), fa.cache_read_int4(*dev[1:7], 3000)
    assert not torch.equal(after[0], want[0]) and not torch.equal(after_read[0], want_read[0])
    for _ in range(5):
        q.zero_()
        lens.zero_()
        for t, f in zip(dev[1:5], fresh):
            t.copy_(f)
        torch.cuda.synchronize()
        fa.rope(x, None, plan, out_q=big)  # long enough for the next launches to queue behind it
        fa.rope(dev[0], None, fa.RopePlan(2, plan.freq, 1.0), offset=0, out_q=q)  # position 0: a copy
        fa.paged_update(lens, dev[6], dev[5].clone(), torch.zeros(400, dtype=torch.int32, device="cuda"),
                        torch.tensor([0, 400], dtype=torch.int32, device="cuda"), 16, max_tokens=4500, seq_lens_out=lens)
        fa.cache_append_int4(rows, rows, slots, *dev[1:5])
        got = fa.decode_paged_int4(q, *dev[1:6], lens, 3000)
        read = fa.cache_read_int4(*dev[1:6], lens, 3000)
        torch.cuda.synchronize()
        for a, b in zip(got + read, after + after_read):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ the step as it is used

@pytest.mark.parametrize("dtype,H,Hkv,d,group,bs", [(torch.bfloat16, 8, 2, 128, 32, 16), (torch.float16, 4, 4, 64, 64, 32),
                                                    (torch.bfloat16, 4, 1, 256, 64, 64)])
def test_prompts_then_decode_steps_then_a_prompt_over_what_was_read_back(dtype, H, Hkv, d, group, bs):
    """Prompts of ragged lengths go in, then tokens one by one from a captured step, with one request idle from
    the middle on.  The cache holds what appending each request's rotated rows gives, the outputs are the
    attention over it, and the forward over the rows read back agrees with them."""
    B, M, steps = 3, 6, 2 * bs + 3
    pool = 14
    g = torch.Generator(device="cuda").manual_seed(d)
    plan = fa.rope_plan(d)
    new = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    lens, table, state = new(B), new(B, M) - 1, torch.tensor([0, pool], dtype=torch.int32, device="cuda")
    ring = torch.randperm(pool, device="cuda", generator=g).int()
    cache = fa.int4_cache(pool, Hkv, bs, d, group)
    prompt = [bs + 3, 1, 2 * bs]
    T = sum(prompt) + 5
    x = torch.randn(T, H + 2 * Hkv, d, device="cuda", generator=g).to(dtype)
    step = fa.paged_update(lens, torch.tensor(prompt, dtype=torch.int32, device="cuda"), table, ring, state, bs,
                           max_tokens=T, seq_lens_out=lens, ring_state_out=state)
    q, k = fa.rope(x[None, :, :H].transpose(1, 2), x[None, :, H:H + Hkv].transpose(1, 2), plan, positions=step.positions)
    fa.cache_append_int4(k[0].transpose(0, 1), x[:, H + Hkv:], step.slot_map, *cache)
    history = [[(k[0, :, t], x[t, H + Hkv:]) for t in range(sum(prompt[:b]), sum(prompt[:b + 1]))] for b in range(B)]

    # one step, captured: lengths and ring state move on in place
    delta, xs = new(B) + 1, torch.zeros(B, H + 2 * Hkv, 1, d, dtype=dtype, device="cuda")
    slots, pos, status = new(B, 1), new(B, 1), new(B)
    qr, kr = torch.empty(B, H, 1, d, dtype=dtype, device="cuda"), torch.empty(B, Hkv, 1, d, dtype=dtype, device="cuda")

    def one():
        fa.paged_update(lens, delta, table, ring, state, bs, seq_lens_out=lens, ring_state_out=state,
                        slot_map=slots.view(-1), positions=pos.view(-1), status=status, rows_per_request=1)
        fa.rope(xs[:, :H], xs[:, H:H + Hkv], plan, positions=pos, out_q=qr, out_k=kr)
        fa.cache_append_int4(kr[:, :, 0], xs[:, H + Hkv:, 0], slots.view(-1), *cache)
        return fa.decode_paged_int4(qr, *cache, table, lens, M * bs, mask="causal")

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = one()
    name = inputs.BF16 if dtype == torch.bfloat16 else inputs.FP16
    for i in range(steps):
        xs.copy_(torch.randn(xs.shape, device="cuda", generator=g))
        if i == bs:
            delta[0] = 0
        graph.replay()
        torch.cuda.synchronize()
        assert status.tolist() == [0, 0, 0]
        for b in range(B):
            if int(delta[b]):
                history[b].append((kr[b, :, 0].clone(), xs[b, H + Hkv:, 0].clone()))
        if i in (0, bs - 1, bs, steps - 1):
            host = [t.cpu().numpy() for t in cache]
            p = dict(q=qr.view(torch.int16).cpu().numpy().view(np.uint16), kc=host[0], vc=host[1], kw=host[2], vw=host[3],
                     table=table.cpu().numpy(), lens=lens.cpu().numpy(), bs=bs, dtype=name)
            _check(p, o, lse, "causal", M * bs)
            assert lens.tolist() == [len(h) for h in history]
            for b in range(B):
                n = len(history[b])
                for codes, words, which in ((host[0], host[2], 0), (host[1], host[3], 1)):
                    want = np.stack([h[which].double().cpu().numpy() for h in history[b]])  # [n, Hkv, d]
                    at = np.array([p["table"][b, j // bs] * bs + j % bs for j in range(n)])
                    wc, ww = ref.append(want, at, np.zeros_like(codes), np.zeros_like(words), bs, group)
                    blocks = np.unique(at // bs)
                    got = ref.gathered(codes, words, p["table"][b], n, bs)
                    assert np.array_equal(got, ref.gathered(wc, ww, p["table"][b], n, bs)) and len(blocks)

    # the rows read back, as the forward takes them: the last row of each request sees what its decode step saw
    S = max(len(h) for h in history)
    kk, vv = fa.cache_read_int4(*cache, table, lens, S, dtype=dtype)
    for b in range(1, B):
        n = len(history[b])
        qq = torch.zeros(1, H, n, d, dtype=dtype, device="cuda")
        qq[:, :, n - 1] = qr[b, :, 0]
        of, lf = fa.forward(qq, kk[b:b + 1, :, :n].contiguous(), vv[b:b + 1, :, :n].contiguous(), mask="causal")
        # both sides are off by roundings of their 16-bit weights, K, V and outputs: 2^-8 each in bf16, of values up to
        # about 4, over few keys
        u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
        assert float((of[0, :, n - 1].float() - o[b, :, 0].float()).abs().max()) <= 16 * u
        assert float((lf[0, :, n - 1] - lse[b, :, 0]).abs().max()) <= 16 * u


def test_every_call_on_another_stream_than_its_tensors():
    p = _problem(2, 8, 2, 1, 128, 32, 16, [300, 40], inputs.BF16, seed=60)
    dev = _device(p)
    k = torch.randn(5, 2, 128, device="cuda").bfloat16()
    slots = torch.arange(5, dtype=torch.int32, device="cuda") + int(dev[5][0, 0]) * 16
    caches = [[t.clone() for t in dev[1:5]] for _ in range(2)]
    fa.cache_append_int4(k, k, slots, *caches[0])
    want = fa.decode_paged_int4(dev[0], *caches[0], *dev[5:], 300) + fa.cache_read_int4(*caches[0], *dev[5:], 300)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    fa.cache_append_int4(k, k, slots, *caches[1], stream=side)
    got = fa.decode_paged_int4(dev[0], *caches[1], *dev[5:], 300, stream=side) + \
        fa.cache_read_int4(*caches[1], *dev[5:], 300, stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
