"""Attention over the 4-bit paged cache where V's scales or the scores of one request lie far apart: what a row
has summed stays right, and finite, wherever its references move."""
import numpy as np
import pytest

import int4_reference as ref
import test_fa_gpu_int4 as base
from exact_io_aware_30_gb300 import fa, inputs

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

_problem, _device = base._problem, base._device

# H, Sq, d, group with one K/V head: 4, 8, 16, 32 and 40 rows
ROWS = [(1, 4, 128, 32), (1, 4, 64, 64), (2, 4, 128, 64), (2, 4, 256, 32), (4, 4, 64, 32), (4, 4, 256, 64), (8, 4, 128, 32),
        (8, 4, 256, 32), (10, 4, 256, 64)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from exact_io_aware_30_gb300 import build
    build.build()
    fa.load()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    assert fa.device_error() == fa.FA_OK


def _known(n, H, Sq, d, group, dtype, scores, v_scale, seed):
    """One request of n tokens and one K/V head.  Every row's score for key j is scores[j] (natural logarithm's
    units; rounded to 15 bf16 steps), every V scale of key j v_scale[j] (a power of two); V's codes and zeros are
    random, no value 0."""
    p = _problem(1, H, 1, Sq, d, group, 16, [n], dtype, seed=seed, junk=False)
    rng = np.random.default_rng(seed)
    q = np.zeros((1, H, Sq, d), np.float32)
    q[..., 0] = 1.0
    p["q"] = inputs.to_bits(q, dtype)
    s = (np.abs(np.asarray(scores, np.float32)) / 15).view(np.uint32) & np.uint32(0xFFFF0000)
    for j in range(n):
        block, at = p["table"][0, j // 16], j % 16
        p["kw"][block, 0, at] = 0
        p["kc"][block, 0, at] = 0x00 if scores[j] >= 0 else 0xFF   # (a group's other values are 0)
        p["kc"][block, 0, at, 0] ^= 0x0F
        p["kw"][block, 0, at, 0] = ref.words(s[j:j + 1].view(np.float32), [0.0 if scores[j] >= 0 else 15.0])[0]
        p["vw"][block, 0, at] = ref.words(np.full(d // group, v_scale[j], np.float32),
                                          rng.choice([-1.0, 16.0], d // group))
    return p


def _check(p, o, lse, mask, max_len, n):
    """The bounds of the attention's tests with V's scales far apart: 2^-11 for a weight's rounding, 2^-15 and n
    2^-23 for the smallest steps of the weights' products, the scores' 2^-18 of their parts, and one rounding of
    O, all relative to what a row sums -- nothing here is absolute but half of the type's smallest step.  What a
    row has summed may in addition have been below fp32's normal numbers, with 11 bits left at least: 2^-11."""
    q = inputs.bits_to_f64(p["q"], p["dtype"])
    want, want_lse, spread, reach, big = ref.decode(q, p["kc"], p["vc"], p["kw"], p["vw"], p["table"], p["lens"],
                                                    max_len, 1.0, mask, p["bs"])
    assert np.all(np.isfinite(want_lse))
    err = np.abs(lse.double().cpu().numpy() - want_lse)
    tol = 2.0 ** -18 * reach + 2.0 ** -20 * (1 + np.abs(want_lse))
    assert np.all(err <= tol), float((err / tol).max())
    least = 2.0 ** -25 if p["dtype"] == inputs.FP16 else 2.0 ** -134
    bound = (2.0 ** -10 + 2 * tol[..., None]) * spread + (2.0 ** -15 + n * 2.0 ** -23) * big + \
        base.U[p["dtype"]] * np.abs(want) + least
    got = o.double().cpu().numpy()
    most = 65504.0 if p["dtype"] == inputs.FP16 else 3.3895e38
    over = np.isinf(got) & (np.sign(got) == np.sign(want)) & (np.abs(want) + bound > most)  # past the type's largest
    err = np.abs(np.where(over, want, got) - want)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
@pytest.mark.parametrize("H,Sq,d,group", ROWS)
@pytest.mark.parametrize("low,high", [(-112, 20), (-114, 100), (-60, 40)])
def test_rows_that_do_not_see_the_key_whose_scale_is_far_larger(low, high, H, Sq, d, group, dtype):
    # keys 128 and later stand in a step of their own, and the draft's earlier rows see none of them
    n = 129
    scale = np.where(np.arange(n) < 128, 2.0 ** low, 2.0 ** high)
    p = _known(n, H, Sq, d, group, dtype, np.linspace(-1, 1, n), scale, H + d)
    o, lse = fa.decode_paged_int4(*_device(p), n, scale=1.0, mask="causal")
    _check(p, o, lse, "causal", n, n)


@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
@pytest.mark.parametrize("H,Sq,d,group", ROWS)
@pytest.mark.parametrize("scales,falls", [((-114, -43, 28, 99), 140.0), ((-114, -43, 28, 99), 60.0), ((-100, 10, -100, 20), 80.0),
                                          ((-30, 34, 98, 110), 100.0), ((0, 30, 60, 90), 30.0), ((-114, 113, -114, 113), 20.0)])
def test_scores_that_fall_while_scales_rise(scales, falls, H, Sq, d, group, dtype):
    # tiles of 128 keys; the first keys of each have its scale and its score
    n = 385
    at = np.arange(n) // 128
    scores = 70.0 - falls * at + np.linspace(0, 1, n)
    p = _known(n, H, Sq, d, group, dtype, scores, 2.0 ** np.array(scales, np.float64)[at], H + d + 1)
    o, lse = fa.decode_paged_int4(*_device(p), n, scale=1.0, mask="none")
    _check(p, o, lse, "none", n, n)


@pytest.mark.parametrize("H,Sq,d,group", ROWS)
@pytest.mark.parametrize("n", [33, 400, 1500])
def test_many_even_keys_with_the_largest_values(n, H, Sq, d, group):
    # a mean of values near the type's largest is finite, although their sum is not
    p = _known(n, H, Sq, d, group, inputs.BF16, np.zeros(n), np.full(n, 2.0 ** 123), n + H)
    p["vw"][:] = ref.words(np.full(d // group, 2.0 ** 123, np.float32), np.zeros(d // group))
    o, lse = fa.decode_paged_int4(*_device(p), n, scale=1.0)
    assert bool(torch.isfinite(o).all())
    _check(p, o, lse, "none", n, n)
