"""Rotary positions on the GPU (fa_rope) against the 64-bit formula: types,
layouts, part of the head, scaled frequencies, far and negative positions,
strided and packed tensors, in place, streams, graphs; the gradient against the
formula's and against differences."""
import numpy as np
import pytest

import step_reference as ref
from exact_io_aware_30_gb300 import fa

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from exact_io_aware_30_gb300 import build
    build.build()
    fa.load()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    assert fa.device_error() == fa.FA_OK


def _f64(t):
    return t.detach().double().cpu().numpy()


def _check(got, x, positions, plan_kw, layout, sign=1.0):
    """Angles: half turns in fp32 below 1, off by at most 2^-25 from rounding and 2^-31 from
    cutting the phase, pi times that in radians, and two steps of sincospi: under 2^-22 in all.
    The products and the sum add 3 half steps of fp32: under 2^-21 of |x1| + |x2|, times the
    amplitude.  Then one rounding to the type (and fp16's smallest step)."""
    f, a = ref.radians(**plan_kw)
    want = ref.rotate(_f64(x), positions, f, a, layout, sign)
    size = ref.rotate(np.abs(_f64(x)), np.zeros_like(positions), f * 0, a, layout)  # a |x|
    rot = 2 * len(f)
    first = np.arange(0, rot // 2) if layout == "half" else np.arange(0, rot, 2)
    second = first + (rot // 2 if layout == "half" else 1)
    both = np.zeros_like(size)
    both[..., first] = both[..., second] = size[..., first] + size[..., second]
    bound = 2.0 ** -21 * both + HALF_STEP[got.dtype] * (np.abs(want) + 2.0 ** -21 * both) + \
        (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    err = np.abs(_f64(got) - want)
    assert np.all(err <= bound), float((err - bound).max())


def _case(B, H, Hkv, S, d, rot, dtype, layout, far=0, seed=0, plan_kw=None, packed=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if packed:
        x = torch.randn(B, S, H + 2 * Hkv, d, device="cuda", generator=g).to(dtype)
        q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hkv].transpose(1, 2)
    else:
        q = torch.randn(B, H, S, d, device="cuda", generator=g).to(dtype)
        k = torch.randn(B, Hkv, S, d, device="cuda", generator=g).to(dtype)
    pos = torch.randint(-far, far + 1, (B, S), device="cuda", generator=g, dtype=torch.int64).int()
    kw = dict(rot=rot, **(plan_kw or {}))
    plan = fa.rope_plan(kw["rot"], **{n: v for n, v in kw.items() if n != "rot"})
    return q, k, pos, kw, plan


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("B,H,Hkv,S,d,rot", [
    (1, 1, 1, 1, 2, 2), (2, 3, 1, 5, 64, 64), (1, 4, 2, 33, 80, 24), (3, 2, 2, 7, 128, 64), (1, 8, 2, 130, 256, 256),
    (2, 5, 5, 3, 18, 6), (1, 2, 1, 9, 1024, 1000), (1, 40, 8, 257, 128, 128), (1, 2, 2, 4, 66, 34)])
def test_against_the_formula(B, H, Hkv, S, d, rot, dtype, layout):
    q, k, pos, kw, plan = _case(B, H, Hkv, S, d, rot, dtype, layout, far=100000, seed=S)
    oq, ok = fa.rope(q, k, plan, positions=pos, layout=layout)
    assert oq.is_contiguous() and oq.shape == q.shape and ok.shape == k.shape
    _check(oq, q, pos.cpu().numpy(), kw, layout)
    _check(ok, k, pos.cpu().numpy(), kw, layout)
    bq, bk = fa.rope_backward(q, k, plan, positions=pos, layout=layout)
    _check(bq, q, pos.cpu().numpy(), kw, layout, -1.0)
    _check(bk, k, pos.cpu().numpy(), kw, layout, -1.0)


@pytest.mark.parametrize("plan_kw", [dict(base=5e5), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                     dict(scaling="by_parts", factor=16.0, original_length=4096)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_scaled_frequencies(plan_kw, layout):
    q, k, pos, kw, plan = _case(1, 4, 2, 50, 128, 128, torch.float32, layout, far=1 << 20, seed=5, plan_kw=plan_kw)
    oq, ok = fa.rope(q, k, plan, positions=pos, layout=layout)
    _check(oq, q, pos.cpu().numpy(), kw, layout)
    _check(ok, k, pos.cpu().numpy(), kw, layout)


def test_positions_none_offset_shared_and_the_farthest():
    q, k, _, kw, plan = _case(2, 4, 2, 37, 128, 128, torch.float32, "half", seed=6)
    for offset in (0, 5, 1 << 30):
        want = np.arange(37)[None].repeat(2, 0) + offset
        oq, ok = fa.rope(q, k, plan, offset=offset)
        _check(oq, q, want, kw, "half")
        _check(ok, k, want, kw, "half")
    row = torch.tensor([2147483647, -2147483648, 0, -1] + list(range(33)), dtype=torch.int32, device="cuda")
    oq = fa.rope(q, None, plan, positions=row, offset=3)
    # fp64 angles of these positions are themselves off by 2^31 * 2^-53 = 2^-22 radians: the
    # formula is evaluated in extended precision instead
    f, _ = ref.radians(128)
    turns = (row.cpu().numpy().astype(np.longdouble) + 3)[:, None] * (f.astype(np.longdouble) / (2 * np.longdouble(np.pi)))
    if np.finfo(np.longdouble).nmant < 63:
        turns = turns[4:]
    theta = (2 * np.pi * (turns - np.round(turns))).astype(np.float64)
    n = len(theta)
    x, y = _f64(q)[:, :, -n:], _f64(oq)[:, :, -n:]
    c, s = np.cos(theta), np.sin(theta)
    want = np.concatenate([x[..., :64] * c - x[..., 64:] * s, x[..., :64] * s + x[..., 64:] * c], -1)
    # the frequencies f are fp64: 2^-53 of up to 2^31 radians is 2^-22 more
    assert np.max(np.abs(y - want)) <= 2.0 ** -20 * 2 * np.max(np.abs(x))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_packed_in_and_out_and_in_place(dtype, layout):
    q, k, pos, kw, plan = _case(2, 6, 2, 19, 64, 48, dtype, layout, far=999, seed=7, packed=True)
    oq, ok = fa.rope(q, k, plan, positions=pos, layout=layout)
    _check(oq, q, pos.cpu().numpy(), kw, layout)
    # written into a packed tensor
    out = torch.full((2, 19, 10, 64), 7.0, dtype=dtype, device="cuda")
    vq, vk = out[:, :, :6].transpose(1, 2), out[:, :, 6:8].transpose(1, 2)
    fa.rope(q, k, plan, positions=pos, layout=layout, out_q=vq, out_k=vk)
    assert torch.equal(vq, oq) and torch.equal(vk, ok) and bool((out[:, :, 8:] == 7).all())
    # in place inside one packed tensor: the other heads and components stay
    base = q._base
    before = base.clone()
    fa.rope(q, k, plan, positions=pos, layout=layout, out_q=q, out_k=k)
    assert torch.equal(q, oq) and torch.equal(k, ok)
    assert torch.equal(base[:, :, 8:], before[:, :, 8:]) and torch.equal(base[..., 48:], before[..., 48:])


def test_odd_bases_and_strides_agree_with_the_contiguous_call():
    g = torch.Generator(device="cuda").manual_seed(8)
    for dtype in (torch.bfloat16, torch.float32):
        plan = fa.rope_plan(64)
        for shift in (0, 1, 2, 4, 8):
            flat = torch.randn(3 * 5 * 7 * 70 + 16, device="cuda", generator=g).to(dtype)
            q = flat[shift:shift + 3 * 5 * 7 * 70].view(3, 7, 5, 70)[..., :66].transpose(1, 2)
            out = fa.rope(q, None, plan)
            assert torch.equal(out, fa.rope(q.contiguous(), None, plan))
            ref.rotate  # (the formula is checked above)


def test_repeated_inputs_and_gradients():
    # an expanded gradient (as of a sum) has strides 0
    plan = fa.rope_plan(32)
    dq = torch.ones(1, 1, 1, 32, device="cuda").expand(2, 3, 11, 32)
    got = fa.rope_backward(dq, None, plan)
    assert torch.equal(got, fa.rope_backward(dq.contiguous(), None, plan))
    with pytest.raises(fa.FAError):
        fa.rope(dq, None, plan, out_q=dq)


def test_gradient_against_differences():
    # the map is linear: <g, rope(x + v) - rope(x)> = <rope_backward(g), v> up to fp32 rounding
    for layout in ("half", "interleaved"):
        q, k, pos, kw, plan = _case(2, 3, 2, 13, 64, 64, torch.float32, layout, far=5000, seed=9,
                                    plan_kw=dict(scaling="by_parts", factor=4.0, original_length=512))
        g, v = torch.randn_like(q), torch.randn_like(q)
        diff = (fa.rope(q + v, None, plan, positions=pos, layout=layout).double() -
                fa.rope(q, None, plan, positions=pos, layout=layout).double())
        left = float((g.double() * diff).sum())
        right = float((fa.rope_backward(g, None, plan, positions=pos, layout=layout).double() * v.double()).sum())
        # each output is within 2^-20 of |x| + |v| (<= 8 here), over n terms of |g| at random signs
        n = q.numel()
        assert abs(left - right) <= 2.0 ** -20 * 16 * float(g.abs().double().sum()) / n ** 0.5 * 4


def test_q_alone_empty_and_refusals():
    plan = fa.rope_plan(64)
    q, k, pos, kw, _ = _case(1, 2, 2, 6, 64, 64, torch.bfloat16, "half", seed=10)
    assert torch.equal(fa.rope(q, None, plan), fa.rope(q, k, plan)[0])
    assert fa.rope(q[:, :, :0], None, plan).shape == (1, 2, 0, 64)
    oq, ok = fa.rope(q, k[:, :0], plan)
    assert ok.shape == (1, 0, 6, 64) and torch.equal(oq, fa.rope(q, None, plan))
    for bad in (lambda: fa.rope(q.double(), None, plan), lambda: fa.rope(q, k.float(), plan),
                lambda: fa.rope(q, k[:, :, :3], plan), lambda: fa.rope(q, None, plan, positions=pos.long()),
                lambda: fa.rope(q, None, plan, positions=pos[:, :3]), lambda: fa.rope(q.cpu(), None, plan),
                lambda: fa.rope(q, None, plan, layout="other"), lambda: fa.rope(q[..., ::2], None, plan),
                lambda: fa.rope(q, None, plan, out_k=k), lambda: fa.rope(q, None, fa.rope_plan(66)),
                lambda: fa.rope(q, None, fa.rope_plan(64, device="cpu")),
                lambda: fa.rope(q, k, plan, out_q=k), lambda: fa.rope(q, k, plan, out_q=q[:, :1].expand_as(q))):
        with pytest.raises(fa.FAError):
            bad()


def test_another_stream_and_a_graph():
    q, k, pos, kw, plan = _case(1, 8, 2, 300, 128, 128, torch.bfloat16, "half", far=70000, seed=11)
    want = fa.rope(q, k, plan, positions=pos)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = fa.rope(q, k, plan, positions=pos, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = fa.rope(q, k, plan, positions=pos, stream=side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.rope(q, k, plan, positions=pos)
    pos.add_(17)
    graph.replay()
    want = fa.rope(q, k, plan, positions=pos)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_past_32_bit_offsets():
    # one head whose rows start 2^31 elements apart
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    big = torch.empty((2 << 31) + 128, dtype=torch.bfloat16, device="cuda")
    q = big.as_strided((1, 1, 3, 128), (0, 0, 1 << 31, 1))
    x = torch.randn(1, 1, 3, 128, device="cuda").bfloat16()
    q.copy_(x)
    plan = fa.rope_plan(128)
    want = fa.rope(x, None, plan)
    assert torch.equal(fa.rope(q, None, plan), want)
    fa.rope(q, None, plan, out_q=q)
    assert torch.equal(q, want)
