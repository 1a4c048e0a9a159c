"""Attention over the 8-bit paged cache on the GPU (fa_decode_paged_fp8)
against the 64-bit formula over the dequantised tokens, and the decode step as
it is used: bookkeeping, rotary positions, append and attention in a row."""
import numpy as np
import pytest

import step_reference as ref
from exact_io_aware_30_gb300 import fa, inputs

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

U = {inputs.BF16: 2.0 ** -8, inputs.FP16: 2.0 ** -11}  # half a step of the type


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
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(
        torch.bfloat16 if dtype == inputs.BF16 else torch.float16).cuda()


def _problem(B, H, Hkv, Sq, d, bs, lens, dtype, seed=0, powers=True, spread=0, junk=True, q_size=1.0):
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
    codes = [inputs.f32_to_e4m3_bits(rng.standard_normal((pool, Hkv, bs, d)) * 100) for _ in range(2)]
    scale = [(2.0 ** rng.integers(-8 - spread, -5 + spread, (pool, Hkv))).astype(np.float32) for _ in range(2)]
    if not powers:
        scale = [s * rng.uniform(1, 2, s.shape).astype(np.float32) for s in scale]
    if junk:  # what no request sees: NaN codes, and scales that are no numbers in the unused blocks
        for b, n in enumerate(lens):
            if n % bs:
                for c in codes:
                    c[table[b, need[b] - 1], :, n % bs:] = rng.choice([0x7F, 0xFF, 0x7E], (Hkv, bs - n % bs, d))
        for block in perm[at:]:
            for c, s in zip(codes, scale):
                c[block], s[block] = 0x7F, np.nan
    qb = inputs.to_bits((rng.standard_normal((B, H, Sq, d)) * q_size).astype(np.float32), dtype)
    return dict(q=qb, kc=codes[0], vc=codes[1], ks=scale[0], vs=scale[1], table=table, lens=lens, bs=bs, dtype=dtype)


def _device(p):
    g = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return [_t16(p["q"], p["dtype"]), g(p["kc"]), g(p["vc"]), g(p["ks"]), g(p["vs"]), g(p["table"]), g(p["lens"])]


def _check(p, o, lse, mask, max_len, scale=None):
    """A weight is rounded to fp16 (2^-11 of it) and then, for bf16, to two e4m3 parts: what the first
    leaves is at most 2^-4 of the weight, what the second leaves 2^-4 of that, 2^-8 in all (three parts
    hold fp16's 11 bits).  Below 2^-14 of the largest of the 256 keys of a step a part's rounding is a
    fixed 2^-22 of that largest (2^-26 with three parts), which over 256 keys of values up to 448 scales
    is 2^-14 (2^-18) of 448 times the largest scale.  The products and sums are fp32: 2^-16 of
    sum p |v| over the lengths here.  O is rounded once.  Scores: a dot of at most 256 exact products
    summed in fp32, 2^-18 of the sum of their sizes, and the exponent's and the logarithm's few steps."""
    d = p["q"].shape[-1]
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    q = inputs.bits_to_f64(p["q"], p["dtype"])
    want, want_lse, spread, reach = ref.decode(q, p["kc"], p["vc"], p["ks"], p["vs"], p["table"], p["lens"], max_len,
                                               scale, mask, p["bs"])
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    u = U[p["dtype"]]
    none = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(lse), none) and np.all(o[none] == 0)
    tol = 2.0 ** -18 * reach + 2.0 ** -20 * (1 + np.abs(np.where(none, 0, want_lse)))
    assert np.all(np.abs(np.where(none, 0, lse) - np.where(none, 0, want_lse)) <= tol)
    vmax = 448.0 * np.nanmax(np.where(np.isfinite(p["vs"]), np.abs(p["vs"]), 0))
    weight = 2.0 ** -11 + (2.0 ** -8 if p["dtype"] == inputs.BF16 else 0.0)
    bound = (weight + 2.0 ** -16 + 2 * tol[..., None]) * spread + u * np.abs(want) + \
        (2.0 ** -14 if p["dtype"] == inputs.BF16 else 2.0 ** -18) * vmax + 2.0 ** -24
    err = np.abs(o - want)
    assert np.all(err <= bound), float((err / bound).max())
    return float((err / bound).max())


CASES = [
    # B, H, Hkv, Sq, d, bs, lens
    (1, 1, 1, 1, 64, 16, [1]),
    (1, 1, 1, 1, 128, 16, [16]),
    (3, 4, 4, 1, 128, 16, [17, 1, 130]),
    (2, 8, 2, 1, 128, 64, [128, 129]),
    (2, 5, 5, 2, 64, 32, [127, 300]),
    (2, 6, 2, 3, 256, 128, [255, 384]),
    (2, 32, 4, 1, 256, 64, [700, 1]),
    (2, 16, 2, 5, 128, 32, [333, 64]),
    (1, 128, 1, 1, 128, 16, [500]),
    (1, 64, 1, 2, 64, 128, [1000]),
    (2, 7, 1, 9, 256, 16, [77, 513]),
    (5, 3, 3, 1, 128, 128, [0, 5, 0, 128, 4000]),
    (1, 2, 2, 1, 64, 16, [9000]),
    (1, 8, 1, 4, 128, 64, [6001]),
]


@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
@pytest.mark.parametrize("mask", ["causal", "none"])
@pytest.mark.parametrize("case", CASES)
def test_against_the_formula(case, mask, dtype):
    p = _problem(*case, dtype, seed=sum(case[:6]))
    max_len = max(1, int(p["lens"].max()))
    o, lse = fa.decode_paged_fp8(*_device(p), max_len, mask=mask)
    _check(p, o, lse, mask, max_len)


@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scales_of_any_value_and_far_apart(d, dtype):
    p = _problem(3, 8, 2, 1, d, 16, [500, 77, 1200], dtype, seed=d, powers=False)
    o, lse = fa.decode_paged_fp8(*_device(p), 1200)
    _check(p, o, lse, "none", 1200)
    p = _problem(2, 4, 1, 2, d, 32, [400, 60], dtype, seed=d + 1, spread=6)
    o, lse = fa.decode_paged_fp8(*_device(p), 400, mask="causal")
    _check(p, o, lse, "causal", 400)
    p = _problem(2, 4, 1, 2, d, 32, [400, 60], dtype, seed=d + 2)
    p["vs"][:] = 0.0
    o, lse = fa.decode_paged_fp8(*_device(p), 400)
    _check(p, o, lse, "none", 400)


@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
def test_score_scale_zero_small_and_large(dtype):
    p = _problem(2, 8, 2, 1, 128, 16, [300, 45], dtype, seed=40)
    for scale in (0.0, 1e-30, 1.0):
        o, lse = fa.decode_paged_fp8(*_device(p), 300, scale=scale)
        _check(p, o, lse, "none", 300, scale)


@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
@pytest.mark.parametrize("size", [1e-4, 30.0])
def test_query_rows_of_very_different_sizes(dtype, size):
    p = _problem(1, 8, 1, 2, 128, 16, [300], dtype, seed=41, q_size=size)
    q = inputs.bits_to_f64(p["q"], dtype)
    q[:, 0] = 0.0
    q[:, 1, :, 1:] = 0.0
    q[:, 2] *= 2.0 ** -6
    q[:, 3, :, 5] = 8.0  # one large component beside small ones
    p["q"] = inputs.to_bits(q.astype(np.float32), dtype)
    o, lse = fa.decode_paged_fp8(*_device(p), 300)
    _check(p, o, lse, "none", 300)


def test_one_outlier_key_before_a_long_even_tail():
    # a spike of weight 1 in the first block, then 20,000 keys of 2^-20: they carry 2 % together
    d, bs, n = 64, 128, 20000
    p = _problem(1, 1, 1, 1, d, bs, [n], inputs.BF16, seed=42, junk=False)
    q = np.zeros((1, 1, 1, d))
    q[..., 0] = 1.0
    p["q"] = inputs.to_bits(q.astype(np.float32), inputs.BF16)
    p["kc"][:] = 0
    p["ks"][:] = 1.0
    p["vs"][:] = 1.0
    p["vc"][:] = inputs.f32_to_e4m3_bits(np.ones(1))[0]
    first = p["table"][0, 0]
    p["kc"][first, 0, 3, 0] = inputs.f32_to_e4m3_bits(np.array([14.0]))[0]
    p["vc"][first, 0, 3] = 0
    o, lse = fa.decode_paged_fp8(*_device(p), n, scale=1.0)
    _check(p, o, lse, "none", n, 1.0)


def test_rows_in_front_of_the_first_token_see_nothing():
    p = _problem(3, 4, 2, 4, 128, 16, [2, 0, 5], inputs.BF16, seed=43)
    o, lse = fa.decode_paged_fp8(*_device(p), 5, mask="causal")
    _check(p, o, lse, "causal", 5)
    assert bool((o[0, :, :2] == 0).all()) and bool(torch.isneginf(lse[1]).all())


def test_lengths_outside_the_bound_are_clamped():
    p = _problem(3, 4, 2, 1, 64, 16, [40, 48, 3], inputs.BF16, seed=44)
    dev = _device(p)
    dev[6] = torch.tensor([1000, -5, 3], dtype=torch.int32, device="cuda")
    o, lse = fa.decode_paged_fp8(*dev, 48)
    p["lens"] = np.array([48, 0, 3], np.int32)
    p["table"][0, :3] = [p["table"][0, 0], p["table"][0, 1], p["table"][0, 2]]
    # request 0's third block now counts to its end: its junk codes must go
    block = p["table"][0, 2]
    p["kc"][block, :, 8:], p["vc"][block, :, 8:] = 0x38, 0x38
    dev[1], dev[2] = torch.from_numpy(p["kc"]).cuda(), torch.from_numpy(p["vc"]).cuda()
    o, lse = fa.decode_paged_fp8(*dev, 48)
    _check(p, o, lse, "none", 48)


def test_blocks_outside_the_pool_read_zeros():
    p = _problem(2, 8, 2, 1, 128, 16, [100, 64], inputs.BF16, seed=45)
    p["table"][0, 1], p["table"][0, 4], p["table"][1, 0] = -1, 10 ** 6, -2 ** 31
    dev = _device(p)
    o, lse = fa.decode_paged_fp8(*dev, 100)
    _check(p, o, lse, "none", 100)


def test_queries_that_are_no_numbers_give_nan_in_their_own_rows_only():
    for dtype, inf, nan in ((inputs.BF16, 0x7F80, 0x7FC0), (inputs.FP16, 0x7C00, 0x7E00)):
        p = _problem(1, 8, 2, 1, 128, 16, [50], dtype, seed=46)
        clean, clean_lse = fa.decode_paged_fp8(*_device(p), 50)
        p["q"][0, 1, 0, 7], p["q"][0, 6, 0, 0] = inf, nan
        o, lse = fa.decode_paged_fp8(*_device(p), 50)
        for h in range(8):
            if h in (1, 6):
                assert bool(torch.isnan(o[0, h]).all()) and bool(torch.isnan(lse[0, h]).all())
            else:
                assert torch.equal(o[0, h], clean[0, h]) and torch.equal(lse[0, h], clean_lse[0, h])


def test_two_calls_give_the_same_bits_and_outputs_can_be_given():
    p = _problem(4, 16, 4, 1, 128, 16, [900, 33, 1, 2000], inputs.FP16, seed=47)
    dev = _device(p)
    a = fa.decode_paged_fp8(*dev, 2000)
    out, lse = torch.empty_like(a[0]), torch.empty_like(a[1])
    st, n = fa.decode_fp8_workspace_query(4, 16, 4, 1, 128, 16, p["table"].shape[1], p["kc"].shape[0], 2000,
                                          dtype=fa.DTYPE_FP16)
    assert st == fa.FA_OK
    ws = torch.full((n + 256,), 0xAB, dtype=torch.uint8, device="cuda")  # its contents do not matter
    b = fa.decode_paged_fp8(*dev, 2000, out=out, lse=lse, workspace=ws)
    assert b[0] is out and torch.equal(a[0], out) and torch.equal(a[1], lse)
    dev[1], dev[2] = dev[1].view(torch.float8_e4m3fn), dev[2].view(torch.float8_e4m3fn)
    c = fa.decode_paged_fp8(*dev, 2000)
    assert torch.equal(a[0], c[0])


def test_two_streams_at_once_and_two_graphs():
    ps = [_problem(4, 8, 2, 1, 128, 16, [900 + i, 33, 1, 2000], inputs.BF16, seed=48 + i) for i in range(2)]
    devs = [_device(p) for p in ps]
    want = [fa.decode_paged_fp8(*d, 2000) for d in devs]
    streams = [torch.cuda.Stream() for _ in devs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [fa.decode_paged_fp8(*d, 2000, stream=s) for d, s in zip(devs, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    graphs, outs = [], []
    for d in devs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(fa.decode_paged_fp8(*d, 2000))
        graphs.append(graph)
    for o, _ in outs:
        o.zero_()
    for _ in range(3):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for g, w in zip(outs, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_refusals():
    p = _problem(2, 8, 2, 1, 128, 16, [50, 20], inputs.BF16, seed=49)
    d = _device(p)
    fa.decode_paged_fp8(*d, 50)

    def with_(i, x):
        return d[:i] + [x] + d[i + 1:]

    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for bad in (lambda: fa.decode_paged_fp8(*with_(0, d[0].float()), 50), lambda: fa.decode_paged_fp8(*with_(0, d[0][:, :7]), 50),
                lambda: fa.decode_paged_fp8(*with_(1, d[1].float()), 50), lambda: fa.decode_paged_fp8(*with_(1, d[1][..., :64]), 50),
                lambda: fa.decode_paged_fp8(*with_(3, d[3].double()), 50), lambda: fa.decode_paged_fp8(*with_(4, d[4][:, :1]), 50),
                lambda: fa.decode_paged_fp8(*with_(5, d[5].long()), 50), lambda: fa.decode_paged_fp8(*with_(6, d[6][:1]), 50),
                lambda: fa.decode_paged_fp8(*with_(6, d[6].cpu()), 50), lambda: fa.decode_paged_fp8(*d, 0),
                lambda: fa.decode_paged_fp8(*d, 65), lambda: fa.decode_paged_fp8(*d, 50, mask="window"),
                lambda: fa.decode_paged_fp8(*d, 50, out=d[0]), lambda: fa.decode_paged_fp8(*d, 50, scale=float("inf")),
                lambda: fa.decode_paged_fp8(*d, 50, lse=torch.empty(2, 8, 1, device="cuda").half()),
                lambda: fa.decode_paged_fp8(*d, 50, workspace=ws[1:])):
        with pytest.raises(fa.FAError):
            bad()


def test_a_cache_of_over_32_bits():
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    bs, Hkv, d, n = 128, 8, 256, 300
    blocks = (1 << 32) // (bs * Hkv * d) + 4
    p = _problem(1, 8, Hkv, 1, d, bs, [n], inputs.BF16, seed=50, junk=False)
    dev = _device(p)
    want = fa.decode_paged_fp8(*dev, n)
    kc = torch.full((blocks, Hkv, bs, d), 0x7F, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    ks, vs = (torch.full((blocks, Hkv), float("nan"), device="cuda") for _ in range(2))
    table = dev[5].clone()
    for i, at in enumerate((blocks - 1, 0, blocks - 2)):
        old = int(dev[5][0, i])
        kc[at], vc[at], ks[at], vs[at] = dev[1][old], dev[2][old], dev[3][old], dev[4][old]
        table[0, i] = at
    got = fa.decode_paged_fp8(dev[0], kc, vc, ks, vs, table, dev[6], n)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("H,Hkv,Sq,d", [(4, 4, 1, 64), (8, 2, 1, 128), (32, 1, 1, 128), (20, 1, 1, 256)])
def test_a_wait_that_runs_out_is_reported_and_the_context_recovers(H, Hkv, Sq, d):
    # one, four, thirty-two and twenty rows per K/V head: the warpgroup shapes
    p = _problem(3, H, Hkv, Sq, d, 16, [700, 3, 129], inputs.BF16, seed=51)
    dev = _device(p)
    assert fa.device_error() == fa.FA_OK
    fa.set_debug_stall_ms(50)
    try:
        fa.decode_paged_fp8(*dev, 700, mask="causal")
        torch.cuda.synchronize()
    finally:
        fa.set_debug_stall_ms(0)
    assert fa.device_error() == fa.FA_ERR_DEVICE_TIMEOUT
    assert fa.device_error() == fa.FA_OK
    o, lse = fa.decode_paged_fp8(*dev, 700, mask="causal")
    _check(p, o, lse, "causal", 700)


@pytest.mark.parametrize("B", [193, 700])
def test_more_requests_than_threads_with_uneven_lengths(B):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 200, B)
    lens[rng.integers(0, B)] = 3000
    p = _problem(B, 2, 1, 1, 64, 16, lens, inputs.BF16, seed=52)
    o, lse = fa.decode_paged_fp8(*_device(p), 3000)
    _check(p, o, lse, "none", 3000)


def test_a_bound_far_above_the_lengths_and_a_wide_table():
    # the grid is sized by the bound; most of its CTAs find no tile
    p = _problem(3, 8, 2, 2, 128, 16, [5, 300, 0], inputs.BF16, seed=53)
    wide = np.full((3, 9000), -1, np.int32)
    wide[:, :p["table"].shape[1]] = p["table"]
    p["table"] = wide
    narrow = fa.decode_paged_fp8(*_device(p), 300, mask="causal")
    o, lse = fa.decode_paged_fp8(*_device(p), 9000 * 16, mask="causal")
    _check(p, o, lse, "causal", 9000 * 16)
    _check(p, *narrow, "causal", 300)


def test_two_host_threads_at_once():
    import threading
    ps = [_problem(3, 8, 2, 1, d, 16, [700, 33, 1200], inputs.FP16, seed=54 + d) for d in (64, 128)]
    devs = [_device(p) for p in ps]
    want = [fa.decode_paged_fp8(*d, 1200) for d in devs]
    torch.cuda.synchronize()
    got, failed = [None, None], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(30):
                got[i] = fa.decode_paged_fp8(*devs[i], 1200, stream=stream)
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
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_the_results_of_the_kernel_in_front_are_seen():
    # the kernels begin before the one in front of them ends: each must still wait for its results
    p = _problem(2, 8, 2, 1, 128, 16, [3000, 1500], inputs.BF16, seed=55)
    dev = _device(p)
    want = fa.decode_paged_fp8(*dev, 3000)
    plan, x = fa.rope_plan(128), torch.randn(1, 64, 8192, 128, device="cuda").bfloat16()
    big, q, lens = torch.empty_like(x), torch.zeros_like(dev[0]), torch.zeros_like(dev[6])
    for _ in range(5):
        q.zero_()
        lens.zero_()
        torch.cuda.synchronize()
        fa.rope(x, None, plan, out_q=big)  # long enough for the next launches to queue behind it
        fa.rope(dev[0], None, fa.RopePlan(2, plan.freq, 1.0), offset=0, out_q=q)  # position 0: a copy
        fa.paged_update(lens, dev[6], dev[5].clone(), torch.zeros(400, dtype=torch.int32, device="cuda"),
                        torch.tensor([0, 400], dtype=torch.int32, device="cuda"), 16, max_tokens=4500, seq_lens_out=lens)
        got = fa.decode_paged_fp8(q, *dev[1:6], lens, 3000)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("n", [300, 3000])
def test_a_graph_with_copies_and_a_fork_in_front(n):
    # copy nodes before the kernels, and a join of two streams before the attention
    p = _problem(2, 8, 2, 1, 128, 16, [n, n // 2], inputs.BF16, seed=56)
    dev = _device(p)
    q, k_new = dev[0].clone(), torch.randn(2, 2, 128, device="cuda").bfloat16()
    slots = torch.tensor([int(dev[5][b, (int(l) - 1) // 16]) * 16 + (int(l) - 1) % 16 for b, l in enumerate(p["lens"])],
                         dtype=torch.int32, device="cuda")
    plan = fa.rope_plan(128)
    fresh = [t.clone() for t in dev[1:5]]

    def step(caches, qin, kin, side):
        qq, kk = torch.empty_like(qin), torch.empty_like(kin)
        qq.copy_(qin)
        q2 = fa.rope(qq, None, plan, offset=7)
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            kk.copy_(kin)
            fa.cache_append_fp8(kk, kk, slots, *caches)
        q3 = fa.rope(q2, None, plan, offset=-7)
        main.wait_stream(side)
        return fa.decode_paged_fp8(q3, *caches, dev[5], dev[6], n) + (q3,)

    side = torch.cuda.Stream()
    want = step([t.clone() for t in fresh], q, k_new, side)
    torch.cuda.synchronize()
    caches = [t.clone() for t in fresh]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(caches, q, k_new, side)
    for t, f in zip(caches, fresh):
        t.copy_(f)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ the step as it is used

@pytest.mark.parametrize("dtype,H,Hkv,d,bs", [(torch.bfloat16, 8, 2, 128, 16), (torch.float16, 4, 4, 64, 32),
                                              (torch.bfloat16, 4, 1, 256, 64)])
def test_prompts_then_decode_steps(dtype, H, Hkv, d, bs):
    """Prompts of ragged lengths go in, then tokens one by one from a captured step, with one
    request finished and its blocks taken by another.  The cache holds what appending each request's
    rotated rows one request at a time gives, and the outputs are the attention over it."""
    B, M, steps = 3, 6, 2 * bs + 3
    pool = 14
    g = torch.Generator(device="cuda").manual_seed(d)
    plan = fa.rope_plan(d)
    new = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    lens, table, state = new(B), new(B, M) - 1, torch.tensor([0, pool], dtype=torch.int32, device="cuda")
    ring = torch.randperm(pool, device="cuda", generator=g).int()
    kc, vc = (torch.full((pool, Hkv, bs, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pool, Hkv), float("nan"), device="cuda") for _ in range(2))
    prompt = [bs + 3, 1, 2 * bs]
    T = sum(prompt) + 5
    x = torch.randn(T, H + 2 * Hkv, d, device="cuda", generator=g).to(dtype)
    step = fa.paged_update(lens, torch.tensor(prompt, dtype=torch.int32, device="cuda"), table, ring, state, bs,
                           max_tokens=T, seq_lens_out=lens, ring_state_out=state)
    q, k = fa.rope(x[None, :, :H].transpose(1, 2), x[None, :, H:H + Hkv].transpose(1, 2), plan, positions=step.positions)
    fa.cache_append_fp8(k[0].transpose(0, 1), x[:, H + Hkv:], step.slot_map, kc, vc, ks, vs)
    history = [[(k[0, :, t], x[t, H + Hkv:]) for t in range(sum(prompt[:b]), sum(prompt[:b + 1]))] for b in range(B)]

    # one step, captured: lengths and ring state move on in place
    delta, xs = new(B) + 1, torch.zeros(B, H + 2 * Hkv, 1, d, dtype=dtype, device="cuda")
    slots, pos, status = new(B), new(B), new(B)
    qr, kr = torch.empty(B, H, 1, d, dtype=dtype, device="cuda"), torch.empty(B, Hkv, 1, d, dtype=dtype, device="cuda")

    def one():
        fa.paged_update(lens, delta, table, ring, state, bs, seq_lens_out=lens, ring_state_out=state, slot_map=slots,
                        positions=pos, status=status)
        fa.rope(xs[:, :H], xs[:, H:H + Hkv], plan, positions=pos[:, None], out_q=qr, out_k=kr)
        fa.cache_append_fp8(kr[:, :, 0], xs[:, H + Hkv:, 0], slots, kc, vc, ks, vs)
        return fa.decode_paged_fp8(qr, kc, vc, ks, vs, table, lens, M * bs, mask="causal")

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = one()
    for i in range(steps):
        xs.copy_(torch.randn(xs.shape, device="cuda", generator=g))
        if i == bs:  # request 0 is done; its slot is empty from here on
            fa.paged_update(lens, torch.tensor([-10 ** 6, 0, 0], dtype=torch.int32, device="cuda"), table, ring, state,
                            bs, max_tokens=0, seq_lens_out=lens, ring_state_out=state)
            history[0] = []
            delta[0] = 0
        graph.replay()
        torch.cuda.synchronize()
        assert status.tolist() == [0, 0, 0]
        rows = iter(range(B))
        for b in range(B):
            if int(delta[b]):
                t = next(rows)
                # row t of slots and positions is request b's: the rows are packed, as rope and append
                # were given them, so request b's new row is xs[t]
                history[b].append((kr[t, :, 0].clone(), xs[t, H + Hkv:, 0].clone()))
        if i in (0, bs - 1, bs, steps - 1):
            name = inputs.BF16 if dtype == torch.bfloat16 else inputs.FP16
            p = dict(q=qr.view(torch.int16).cpu().numpy().view(np.uint16), kc=kc.cpu().numpy(), vc=vc.cpu().numpy(),
                     ks=ks.cpu().numpy(), vs=vs.cpu().numpy(), table=table.cpu().numpy(), lens=lens.cpu().numpy(), bs=bs,
                     dtype=name)
            _check(p, o, lse, "causal", M * bs)
            assert lens.tolist() == [len(h) for h in history]
            for b in range(B):
                n = len(history[b])
                for cache, scale, which in ((p["kc"], p["ks"], 0), (p["vc"], p["vs"], 1)):
                    if not n:
                        continue
                    got = ref.gathered(cache, scale, p["table"][b], n, bs)
                    want = np.stack([h[which].double().cpu().numpy() for h in history[b]], 1)
                    for j in range(0, n, bs):
                        s = scale[p["table"][b, j // bs]].astype(np.float64)[:, None, None]
                        # a code is within half a step, 2^-4 of the value or 2^-10 of the scale, and each
                        # growth of the scale while the block filled may have added half of 2^-9 of it
                        tol = 2.0 ** -4 * np.abs(want[:, j:j + bs]) + 2.0 ** -9 * s
                        assert np.all(np.abs(got[:, j:j + bs] - want[:, j:j + bs]) <= tol)
