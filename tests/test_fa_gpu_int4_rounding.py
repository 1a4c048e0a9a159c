"""Attention over the 4-bit paged cache: what a weight's rounding and the sums of very long requests leave of O."""
import numpy as np
import pytest

import int4_reference as ref
import test_fa_gpu_int4 as base
from exact_io_aware_30_gb300 import fa, inputs

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

_problem, _device, _dev, _t16 = base._problem, base._device, base._dev, base._t16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from exact_io_aware_30_gb300 import build
    build.build()
    fa.load()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    assert fa.device_error() == fa.FA_OK


def _check_fine(p, o, lse, max_len, scale, mask="none"):
    """With fp16, and up to four rows per K/V head in bf16 too, a weight times its scale is held in two fp16 numbers, 2^-22 of it; the second's
    smallest half step is 2^-25, no more than that of a product of 2^-3 or more, 2^9 below a row's largest (2^6 at
    least when it is summed), and here all lie nearer.  The rest as in the attention's other tests: the scores', the
    sums' 2^-17 of sum p s (15 + |z|) (2^-23 of what is held at each of at most 64 products), and one rounding of O."""
    q = inputs.bits_to_f64(p["q"], p["dtype"])
    want, want_lse, spread, reach, big = ref.decode(q, p["kc"], p["vc"], p["kw"], p["vw"], p["table"], p["lens"],
                                                    max_len, scale, mask, p["bs"])
    tol = 2.0 ** -18 * reach + 2.0 ** -20 * (1 + np.abs(want_lse))
    err = np.abs(lse.double().cpu().numpy() - want_lse)
    assert np.all(err <= tol), float((err / tol).max())
    bound = (2.0 ** -22 + 2 * tol[..., None]) * spread + 2.0 ** -17 * big + base.U[p["dtype"]] * np.abs(want)
    if p["dtype"] == inputs.FP16:
        bound = bound + 2.0 ** -25
    err = np.abs(o.double().cpu().numpy() - want)
    assert np.all(err <= bound), float((err / bound).max())


def _scores(p, scores):
    """Every row's scores by token, |score| <= 15 steps of bf16 (scale 1): q is the first unit vector."""
    q = np.zeros(p["q"].shape, np.float32)
    q[..., 0] = 1.0
    p["q"] = inputs.to_bits(q, p["dtype"])
    bs = p["bs"]
    for b, L in enumerate(p["lens"]):
        for j in range(int(L)):
            block, at = p["table"][b, j // bs], j % bs
            p["kw"][block, :, at], p["kc"][block, :, at] = 0, 0
            p["kc"][block, :, at, 0] = 0x0F
            p["kw"][block, :, at, 0] = ref.words(inputs.bits_to_f64(inputs.to_bits(
                np.array([scores[j] / 15], np.float32), inputs.BF16), inputs.BF16).astype(np.float32), [0.0])[0]


def _cancel(p):
    """V of each request's second key becomes that of its first with the sign turned: O is the difference of two
    weights times V, and a weight rounded to 11 bits would be seen in it."""
    for b in range(len(p["lens"])):
        block = p["table"][b, 0]
        p["vc"][block, :, 1] = 0xFF - p["vc"][block, :, 0]
        s, z = ref.unpack_words(p["vw"][block, :, 0])
        p["vw"][block, :, 0] = ref.words(s, np.rint(z))
        p["vw"][block, :, 1] = ref.words(s, 15 - np.rint(z))


@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
@pytest.mark.parametrize("H,Hkv,Sq", [(2, 2, 1), (4, 2, 1), (4, 1, 1), (2, 2, 4)])
@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (256, 32), (256, 64)])
def test_up_to_four_rows_two_keys_that_nearly_cancel(d, group, H, Hkv, Sq, dtype):
    p = _problem(8, H, Hkv, Sq, d, group, 16, [2] * 8, dtype, seed=d + H, q_size=0.002)
    _cancel(p)
    o, lse = fa.decode_paged_int4(*_device(p), 2)
    _check_fine(p, o, lse, 2, 1 / np.sqrt(d))


@pytest.mark.parametrize("H,Hkv,Sq", [(5, 1, 1), (16, 2, 1), (16, 1, 1), (8, 1, 4), (8, 1, 5)])
@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (256, 32), (256, 64)])
def test_fp16_more_rows_two_keys_that_nearly_cancel(d, group, H, Hkv, Sq):
    p = _problem(8, H, Hkv, Sq, d, group, 16, [2] * 8, inputs.FP16, seed=d + H, q_size=0.002)
    _cancel(p)
    o, lse = fa.decode_paged_int4(*_device(p), 2)
    _check_fine(p, o, lse, 2, 1 / np.sqrt(d))


ROWS = [(4, 1, inputs.BF16), (4, 1, inputs.FP16), (8, 1, inputs.FP16), (16, 1, inputs.FP16), (16, 2, inputs.FP16), (8, 5, inputs.FP16)]


@pytest.mark.parametrize("H,Sq,dtype", ROWS)
@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (256, 32), (256, 64)])
@pytest.mark.parametrize("n", [1, 7, 40, 129, 520])
def test_few_keys(n, d, group, H, Sq, dtype):
    p = _problem(3, H, 1, Sq, d, group, 16, [n, max(1, n - 1), n], dtype, seed=n + d, q_size=0.05)
    o, lse = fa.decode_paged_int4(*_device(p), n)
    _check_fine(p, o, lse, n, 1 / np.sqrt(d))


@pytest.mark.parametrize("H,Sq,dtype", ROWS)
@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (256, 32), (256, 64)])
@pytest.mark.parametrize("rise", [6.0, 9.0])
def test_references_that_move(rise, d, group, H, Sq, dtype):
    # a key in every 32 carries the weight, and those of a tile lie above those of the tile in front, so that all
    # sums are rescaled (the rest of the weights too); the last tile's values are 0, so that O is what the tiles in
    # front of it left
    n = 4 * 128
    p = _problem(1, H, 1, Sq, d, group, 16, [n], dtype, seed=d, junk=False)
    _scores(p, np.where(np.arange(n) % 32 == 0, 20.0 + rise * (np.arange(n) // 128), 0.0))
    for j in range(n - 128, n):
        block, at = p["table"][0, j // 16], j % 16
        p["vc"][block, 0, at] = 0x88
        p["vw"][block, 0, at] = ref.words(np.ones(d // group, np.float32), np.full(d // group, 8.0))
    o, lse = fa.decode_paged_int4(*_device(p), n, scale=1.0)
    _check_fine(p, o, lse, n, 1.0)


@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
@pytest.mark.parametrize("H,d,group", [(2, 128, 32), (4, 64, 64), (8, 128, 64), (32, 256, 32)])
@pytest.mark.parametrize("down", [14.0, 17.0, 20.0])
def test_a_first_key_that_outweighs_very_many_even_ones(down, H, d, group, dtype):
    """Key 0 stands `down` (natural logarithm) above 131,071 even keys, whose table names one block again and again.
    Their products lie 1.44 down below the row's largest: of the keys that share a warp's references with key 0, at
    most 4,096, each is off by at most 2^-31 of that (2^-37, 6 ahead); the others' references are their own.  Beside
    it a weight's 2^-11, the scores' share, 2^-15 of the sums, and one rounding of O."""
    n, bs = 1 << 17, 128
    rng = np.random.default_rng(int(down) + H)
    p = _problem(1, H, 1, 1, d, group, bs, [2 * bs], dtype, seed=H, junk=False)
    _scores(p, np.where(np.arange(2 * bs) == 0, down, 0.0))
    table = np.full((1, n // bs), p["table"][0, 1], np.int32)
    table[0, 0] = p["table"][0, 0]
    dev = _device(p)
    dev[5], dev[6] = _dev(table), _dev(np.array([n], np.int32))
    o, lse = fa.decode_paged_int4(*dev, n, scale=1.0)
    v = ref.gathered(p["vc"], p["vw"], p["table"][0], 2 * bs, bs)[0]
    k = ref.gathered(p["kc"], p["kw"], p["table"][0], 2 * bs, bs)[0]
    top = k[0, 0]
    w = np.exp(k[:, 0] - top) * np.where(np.arange(2 * bs) < bs, 1, n // bs - 1)
    want, spread, total = w @ v / w.sum(), w @ np.abs(v) / w.sum(), top + np.log(w.sum())
    s, z = [np.concatenate([x[int(p["table"][0, i]), 0] for i in range(2)]) for x in ref.unpack_words(p["vw"])]
    size = np.repeat(s * (15 + np.abs(z)), group, -1)
    big = w @ size / w.sum()
    tol = 2.0 ** -18 * 2 * top + 2.0 ** -20 * (1 + total)
    assert float((lse.double() - total).abs().max()) <= tol
    bound = (2.0 ** -11 + 2 * tol) * spread + 2.0 ** -15 * big + 4096 * 2.0 ** -31 * size.max(0) + base.U[dtype] * np.abs(want) + 2.0 ** -25
    err = np.abs(o.double().cpu().numpy()[0, :, 0] - want)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("H,d,group,n", [(32, 256, 32, 1 << 20), (32, 128, 64, 1 << 20), (16, 256, 64, 1 << 20), (8, 64, 32, 1 << 21),
                                         (4, 128, 32, 1 << 21)])
def test_sums_over_very_long_requests_whose_codes_are_large(H, d, group, n):
    """A unit per CTA, of so many keys that a sum cut off at each of their products, by up to 2^-23 of what it holds,
    could lose 2^-8 of itself.  All codes are near 15.  The sums are allowed 2^-15 of sum p s (15 + |z|) (at most 512
    products in a row, 2^-23 of what is held at each, and 512 pieces of them), those of the weights 2^-15 (512 in a row
    and 512 pieces, 2^-25 each on the mean), a weight 2^-11 of its value, and the scores' share as in the other tests."""
    B, bs = 152 * 3, 128
    rng = np.random.default_rng(H + d)
    p = _problem(1, H, 1, 1, d, group, bs, [bs], inputs.FP16, seed=d, junk=False, q_size=0.02)
    p["vc"][:] = ref.pack(rng.integers(14, 16, (*p["vc"].shape[:-1], d)))
    s, _ = ref.unpack_words(p["vw"])
    p["vw"][:] = ref.words(s, rng.integers(7, 9, s.shape))
    want, want_lse, spread, reach, big = [x[0, :, 0] for x in ref.decode(
        inputs.bits_to_f64(p["q"], inputs.FP16), p["kc"], p["vc"], p["kw"], p["vw"], p["table"], p["lens"], bs,
        1 / np.sqrt(d), "none", bs)]
    dev = _device(p)
    table = torch.full((1, n // bs), int(p["table"][0, 0]), dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    q = dev[0].expand(B, -1, -1, -1).contiguous()
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    o, lse = fa.decode_paged_int4(q, *dev[1:5], table, lens, n)
    want_lse = want_lse + np.log(n // bs)  # the same keys again and again
    tol = 2.0 ** -18 * reach + 2.0 ** -20 * (1 + np.abs(want_lse)) + 2.0 ** -15
    assert np.all(np.abs(lse[..., 0].double().cpu().numpy() - want_lse) <= tol)
    bound = (2.0 ** -11 + 2 * tol[:, None]) * spread + 2.0 ** -15 * big + base.U[inputs.FP16] * np.abs(want)
    err = np.abs(o[:, :, 0].double().cpu().numpy() - want)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("mask", ["causal", "none"])
@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
@pytest.mark.parametrize("H,Hkv,Sq,d,group,n", [(32, 4, 4, 256, 32, 1 << 20), (16, 4, 1, 128, 32, 1 << 21), (64, 4, 1, 128, 64, 1 << 21),
                                                (32, 4, 1, 64, 32, 1 << 21), (40, 4, 4, 128, 32, 1 << 20)])
def test_long_units_that_are_cut_and_rest(H, Hkv, Sq, d, group, n, dtype, mask):
    """Units longer than a CTA's share, and shares longer than sums are kept: partials of pieces.  A second request is
    short.  Each call gives the same bits, replayed from a graph too.  Bounds as above."""
    bs = 128
    lens = [n - 37, 300]
    p = _problem(1, H, Hkv, Sq, d, group, bs, [3 * bs], dtype, seed=H + d, junk=False, q_size=0.02)
    dev = _device(p)
    table = torch.full((2, n // bs), -1, dtype=torch.int32)
    table[0] = torch.from_numpy(p["table"][0])[torch.arange(n // bs) % 3]
    table[1, :3] = torch.from_numpy(p["table"][0])
    q, table = dev[0].expand(2, -1, -1, -1).contiguous(), table.cuda()
    given = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = fa.decode_paged_int4(q, *dev[1:5], table, given, n, mask=mask)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = fa.decode_paged_int4(q, *dev[1:5], table, given, n, mask=mask)
    for _ in range(2):
        graph.replay()
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    k, v = [ref.gathered(p[c], p[w], p["table"][0], 3 * bs, bs) for c, w in (("kc", "kw"), ("vc", "vw"))]
    sizes = []
    for w in ("kw", "vw"):
        s, z = ref.unpack_words(np.concatenate([p[w][int(p["table"][0, i])] for i in range(3)], 1))
        sizes.append(np.repeat(s * (15 + np.abs(z)), group, -1))  # [Hkv, 384, d]
    x = inputs.bits_to_f64(p["q"], dtype)[0]
    for b, L in enumerate(lens):
        for h in range(H):
            g = h // (H // Hkv)
            for i in range(Sq):
                seen = L if mask == "none" else L - Sq + 1 + i
                times = seen // (3 * bs) + (np.arange(3 * bs) < seen % (3 * bs))
                score = x[h, i] @ k[g].T / np.sqrt(d)
                top = score[times > 0].max()
                w = times * np.exp(score - top)
                total = top + np.log(w.sum())
                w = w / w.sum()
                tol = 2.0 ** -18 * (np.abs(x[h, i]) @ sizes[0][g].T).max() / np.sqrt(d) + 2.0 ** -20 * (1 + abs(total)) + 2.0 ** -15
                assert abs(float(lse[b, h, i]) - total) <= tol
                want = w @ v[g]
                bound = (2.0 ** -11 + 2 * tol) * (w @ np.abs(v[g])) + 2.0 ** -15 * (w @ sizes[1][g]) + \
                    base.U[dtype] * np.abs(want) + 2.0 ** -25
                assert np.all(np.abs(o[b, h, i].double().cpu().numpy() - want) <= bound)
