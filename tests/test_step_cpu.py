"""Refusals and host-side parts of the decode step's entry points -- rotary
positions, the paged cache's bookkeeping, the quantising append and decoding
over the 8-bit cache -- without a GPU: every call here fails validation before
it touches the device."""
import ctypes

import numpy as np
import pytest

import step_reference as ref
from exact_io_aware_30_gb300 import build, fa, inputs

FAKE = 0x7F0000001000  # 256-byte aligned, never dereferenced: validation fails first
GB = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return fa.load()


# ------------------------------------------------------------------ rotary frequencies

@pytest.mark.parametrize("rot", [2, 6, 64, 128, 256, 1024])
@pytest.mark.parametrize("kw", [dict(), dict(base=1.0), dict(base=5e5), dict(scaling="linear", factor=4.0),
                                dict(scaling="ntk", factor=8.0),
                                dict(scaling="by_parts", factor=16.0, original_length=4096),
                                dict(scaling="by_parts", factor=2.0, original_length=100, low_turns=0.5,
                                     high_turns=3.0)])
def test_frequencies_are_the_formula_s(rot, kw):
    freq, amplitude = fa.rope_frequencies(rot, **kw)
    f, a = ref.radians(rot, **kw)
    assert len(freq) == rot // 2
    # both sides evaluate a few correctly rounded fp64 steps and one power
    # (its argument's rounding grows by ln(base) <= 37): 64 half steps; the
    # fixed-point frequency is within half a unit of 2^-64 turn
    np.testing.assert_allclose(np.array(freq, dtype=np.float64) * (2 * np.pi) / 2.0 ** 64, f, rtol=64 * 2.0 ** -53,
                               atol=2 * np.pi * 2.0 ** -65)
    assert amplitude == np.float32(a)


def test_ntk_stretches_the_slowest_pair_by_the_factor():
    plain, _ = fa.rope_frequencies(128)
    far, _ = fa.rope_frequencies(128, scaling="ntk", factor=4.0)
    assert far[0] == plain[0]
    assert abs(plain[-1] / far[-1] - 4.0) < 1e-9


@pytest.mark.parametrize("kw,status", [
    (dict(rot_dim=0), fa.FA_ERR_INVALID_ARG), (dict(rot_dim=7), fa.FA_ERR_INVALID_ARG),
    (dict(rot_dim=1026), fa.FA_ERR_INVALID_ARG), (dict(base=0.5), fa.FA_ERR_INVALID_ARG),
    (dict(base=float("nan")), fa.FA_ERR_INVALID_ARG), (dict(scaling="linear", factor=0.5), fa.FA_ERR_INVALID_ARG),
    (dict(scaling="linear", factor=float("inf")), fa.FA_ERR_INVALID_ARG),
    (dict(base=1e308, scaling="ntk", factor=1e300), fa.FA_ERR_INVALID_ARG),
    (dict(scaling="by_parts", factor=2.0), fa.FA_ERR_INVALID_ARG),
    (dict(scaling="by_parts", factor=2.0, original_length=64, low_turns=4.0, high_turns=4.0), fa.FA_ERR_INVALID_ARG),
    (dict(scaling="unknown"), fa.FA_ERR_UNSUPPORTED)])
def test_frequencies_refused(kw, status):
    a = dict(rot_dim=64)
    a.update(kw)
    with pytest.raises(fa.FAError) as e:
        fa.rope_frequencies(**a)
    assert e.value.status == status


# ------------------------------------------------------------------ rope

def _rope(**kw):
    a = dict(q=FAKE, qs=(4096, 128, 512), q_out=FAKE + GB, qos=(4096, 128, 512), k=FAKE + 2 * GB,
             ks=(4096, 128, 512), k_out=FAKE + 3 * GB, kos=(4096, 128, 512), positions=None, pos_stride=0, offset=0,
             freq=FAKE + 4 * GB, amplitude=1.0, B=2, H=4, Hkv=4, S=8, d=128, rot=128, layout=0, direction=0,
             dtype=fa.DTYPE_BF16)
    a.update(kw)
    arr = lambda t: None if t is None else (ctypes.c_longlong * 3)(*t)
    return fa.load().fa_rope(a["q"], arr(a["qs"]), a["q_out"], arr(a["qos"]), a["k"], arr(a["ks"]), a["k_out"],
                             arr(a["kos"]), a["positions"], a["pos_stride"], a["offset"], a["freq"], a["amplitude"],
                             a["B"], a["H"], a["Hkv"], a["S"], a["d"], a["rot"], a["layout"], a["direction"],
                             a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), fa.FA_ERR_UNSUPPORTED), (dict(layout=2), fa.FA_ERR_UNSUPPORTED),
    (dict(direction=2), fa.FA_ERR_INVALID_ARG), (dict(B=0), fa.FA_ERR_INVALID_ARG),
    (dict(H=0), fa.FA_ERR_INVALID_ARG), (dict(Hkv=-1), fa.FA_ERR_INVALID_ARG), (dict(S=-1), fa.FA_ERR_INVALID_ARG),
    (dict(rot=127), fa.FA_ERR_INVALID_ARG), (dict(rot=0), fa.FA_ERR_INVALID_ARG),
    (dict(rot=130), fa.FA_ERR_INVALID_ARG), (dict(d=1026, rot=64), fa.FA_ERR_INVALID_ARG),
    (dict(amplitude=float("inf")), fa.FA_ERR_INVALID_ARG), (dict(q=None), fa.FA_ERR_INVALID_ARG),
    (dict(k=None), fa.FA_ERR_INVALID_ARG), (dict(qs=None), fa.FA_ERR_INVALID_ARG),
    (dict(freq=None), fa.FA_ERR_INVALID_ARG), (dict(qs=(4096, -128, 512)), fa.FA_ERR_INVALID_ARG),
    (dict(qs=(1 << 41, 128, 512)), fa.FA_ERR_INVALID_ARG), (dict(q=FAKE + 1), fa.FA_ERR_MISALIGNED),
    (dict(dtype=fa.DTYPE_FP32, k_out=FAKE + 3 * GB + 2), fa.FA_ERR_MISALIGNED),
    (dict(freq=FAKE + 4 * GB + 4), fa.FA_ERR_MISALIGNED), (dict(positions=FAKE + 5 * GB + 1), fa.FA_ERR_MISALIGNED),
    # outputs whose elements coincide: a repeated head, interleaved rows
    (dict(qos=(4096, 0, 512)), fa.FA_ERR_INVALID_ARG), (dict(kos=(4096, 128, 500)), fa.FA_ERR_INVALID_ARG),
    # an output over another input, over the other output, over the frequencies, over its input but shifted
    (dict(q_out=FAKE + 2 * GB), fa.FA_ERR_INVALID_ARG), (dict(k_out=FAKE + GB), fa.FA_ERR_INVALID_ARG),
    (dict(freq=FAKE + GB), fa.FA_ERR_INVALID_ARG), (dict(q_out=FAKE + 256), fa.FA_ERR_INVALID_ARG),
    (dict(q_out=FAKE, qos=(4096, 512, 128)), fa.FA_ERR_INVALID_ARG),
    (dict(positions=FAKE + GB, pos_stride=8), fa.FA_ERR_INVALID_ARG)])
def test_rope_refused(kw, status):
    assert _rope(**kw) == status


def test_rope_in_place_on_heads_of_one_packed_tensor_passes_the_checks():
    # [B, S, 12 heads, 128]: q heads 0-3, k heads 4-7, v heads 8-11 stay; on a
    # machine without a GPU a call whose arguments are all right ends at the device probe
    st = (8 * 1536, 128, 1536)
    packed = dict(q=FAKE, qs=st, q_out=FAKE, qos=st, k=FAKE + 1024, ks=st, k_out=FAKE + 1024, kos=st)
    ok = _rope()
    assert ok not in (fa.FA_ERR_INVALID_ARG, fa.FA_ERR_MISALIGNED) or ok == fa.FA_OK
    if ok == fa.FA_ERR_CUDA:  # no device here
        assert _rope(**packed) == ok
    # q's last head is k's first
    packed.update(k=FAKE + 768, k_out=FAKE + 768)
    assert _rope(**packed) == fa.FA_ERR_INVALID_ARG


def test_rope_of_no_tokens_is_ok():
    assert _rope(S=0, q=None, k=None, freq=None) == fa.FA_OK


# ------------------------------------------------------------------ paged update

def _update(**kw):
    names = ("seq_lens", "delta", "table", "ring", "state", "lens_out", "state_out", "slots", "positions", "status")
    a = {n: FAKE + i * GB for i, n in enumerate(names)}
    a.update(B=4, max_blocks=8, ring_size=64, bs=16, rows=32)
    a.update(kw)
    return fa.load().fa_paged_update(*[a[n] for n in names], a["B"], a["max_blocks"], a["ring_size"], a["bs"],
                                     a["rows"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(bs=8), fa.FA_ERR_UNSUPPORTED), (dict(bs=0), fa.FA_ERR_UNSUPPORTED), (dict(bs=48), fa.FA_ERR_UNSUPPORTED),
    (dict(B=0), fa.FA_ERR_INVALID_ARG), (dict(max_blocks=0), fa.FA_ERR_INVALID_ARG),
    (dict(ring_size=0), fa.FA_ERR_INVALID_ARG), (dict(rows=-1), fa.FA_ERR_INVALID_ARG),
    (dict(max_blocks=1 << 27, bs=16), fa.FA_ERR_INVALID_ARG), (dict(B=1 << 20, max_blocks=1 << 12), fa.FA_ERR_INVALID_ARG),
    (dict(delta=None), fa.FA_ERR_INVALID_ARG), (dict(slots=None), fa.FA_ERR_INVALID_ARG),
    (dict(ring=FAKE + 3 * GB + 2), fa.FA_ERR_MISALIGNED), (dict(slots=FAKE), fa.FA_ERR_INVALID_ARG),
    (dict(status=FAKE + 7 * GB + 124), fa.FA_ERR_INVALID_ARG), (dict(lens_out=FAKE + 4), fa.FA_ERR_INVALID_ARG),
    (dict(state_out=FAKE), fa.FA_ERR_INVALID_ARG), (dict(table=FAKE + 3 * GB), fa.FA_ERR_INVALID_ARG)])
def test_update_refused(kw, status):
    assert _update(**kw) == status


# ------------------------------------------------------------------ append

def _append(**kw):
    a = dict(k=FAKE, v=FAKE + GB, kt=1024, kh=128, vt=1024, vh=128, slots=FAKE + 2 * GB, kc=FAKE + 3 * GB,
             vc=FAKE + 4 * GB, ks=FAKE + 5 * GB, vs=FAKE + 6 * GB, T=4, Hkv=8, d=128, bs=16, blocks=64,
             dtype=fa.DTYPE_BF16)
    a.update(kw)
    return fa.load().fa_cache_append_fp8(a["k"], a["v"], a["kt"], a["kh"], a["vt"], a["vh"], a["slots"], a["kc"],
                                         a["vc"], a["ks"], a["vs"], a["T"], a["Hkv"], a["d"], a["bs"], a["blocks"],
                                         a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=fa.DTYPE_FP32), fa.FA_ERR_UNSUPPORTED), (dict(d=96), fa.FA_ERR_UNSUPPORTED),
    (dict(bs=24), fa.FA_ERR_UNSUPPORTED), (dict(Hkv=0), fa.FA_ERR_INVALID_ARG), (dict(T=-1), fa.FA_ERR_INVALID_ARG),
    (dict(T=(1 << 30) + 1), fa.FA_ERR_INVALID_ARG),
    (dict(blocks=0), fa.FA_ERR_INVALID_ARG), (dict(blocks=1 << 27), fa.FA_ERR_INVALID_ARG),
    (dict(Hkv=65536), fa.FA_ERR_INVALID_ARG), (dict(v=None), fa.FA_ERR_INVALID_ARG),
    (dict(kt=-1), fa.FA_ERR_INVALID_ARG), (dict(k=FAKE + 1), fa.FA_ERR_MISALIGNED),
    (dict(kc=FAKE + 3 * GB + 8), fa.FA_ERR_MISALIGNED), (dict(vs=FAKE + 6 * GB + 2), fa.FA_ERR_MISALIGNED),
    (dict(kc=FAKE), fa.FA_ERR_INVALID_ARG), (dict(vc=FAKE + 3 * GB + 4096), fa.FA_ERR_INVALID_ARG),
    (dict(ks=FAKE + 3 * GB + 64), fa.FA_ERR_INVALID_ARG), (dict(vs=FAKE + 5 * GB), fa.FA_ERR_INVALID_ARG)])
def test_append_refused(kw, status):
    assert _append(**kw) == status


def test_append_of_no_rows_is_ok():
    assert _append(T=0, k=None, v=None, slots=None) == fa.FA_OK


# ------------------------------------------------------------------ decode over the 8-bit cache

def _decode(**kw):
    a = dict(q=FAKE, kc=FAKE + GB, vc=FAKE + 2 * GB, ks=FAKE + 3 * GB, vs=FAKE + 4 * GB, table=FAKE + 5 * GB,
             lens=FAKE + 6 * GB, o=FAKE + 7 * GB, lse=FAKE + 8 * GB, ws=FAKE + 9 * GB, ws_bytes=GB, B=2, H=8, Hkv=2,
             Sq=1, d=128, bs=16, max_blocks=8, blocks=64, max_len=128, scale=0.1, mask=fa.MASK_CAUSAL,
             dtype=fa.DTYPE_BF16)
    a.update(kw)
    return fa.load().fa_decode_paged_fp8(
        a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["lens"], a["o"], a["lse"], a["ws"], a["ws_bytes"],
        a["B"], a["H"], a["Hkv"], a["Sq"], a["d"], a["bs"], a["max_blocks"], a["blocks"], a["max_len"], a["scale"],
        a["mask"], a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=fa.DTYPE_FP32), fa.FA_ERR_UNSUPPORTED), (dict(d=80), fa.FA_ERR_UNSUPPORTED),
    (dict(bs=256), fa.FA_ERR_UNSUPPORTED), (dict(mask=fa.MASK_SLIDING_WINDOW), fa.FA_ERR_UNSUPPORTED),
    (dict(H=9), fa.FA_ERR_INVALID_ARG), (dict(Hkv=0), fa.FA_ERR_INVALID_ARG), (dict(Sq=0), fa.FA_ERR_INVALID_ARG),
    (dict(Sq=33), fa.FA_ERR_UNSUPPORTED), (dict(max_len=0), fa.FA_ERR_INVALID_ARG),
    (dict(max_len=129), fa.FA_ERR_INVALID_ARG),
    (dict(B=1, max_blocks=1 << 27, max_len=0x7fffffff - 511), fa.FA_ERR_INVALID_ARG), (dict(blocks=0), fa.FA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), fa.FA_ERR_INVALID_ARG), (dict(scale=-0.1), fa.FA_ERR_INVALID_ARG),
    (dict(ks=None), fa.FA_ERR_INVALID_ARG), (dict(kc=FAKE + GB + 8), fa.FA_ERR_MISALIGNED),
    (dict(vs=FAKE + 4 * GB + 1), fa.FA_ERR_MISALIGNED), (dict(ws=FAKE + 9 * GB + 16), fa.FA_ERR_MISALIGNED)])
def test_decode_refused(kw, status):
    assert _decode(**kw) == status


def test_decode_workspace_query_needs_a_place_for_its_answer():
    assert fa.load().fa_decode_fp8_workspace_query(2, 8, 2, 1, 128, 16, 8, 64, 128, 0, 0, None) == fa.FA_ERR_INVALID_ARG
    st, n = fa.decode_fp8_workspace_query(2, 8, 2, 1, 96, 16, 8, 64, 128)
    assert (st, n) == (fa.FA_ERR_UNSUPPORTED, 0)


# ------------------------------------------------------------------ the reference itself

@pytest.mark.parametrize("amax,scale", [(448.0, 1.0), (448.25, 2.0), (1.75, 2.0 ** -8), (1.0, 2.0 ** -8),
                                        (1.7578125, 2.0 ** -7), (0.0, 2.0 ** -126), (2.0 ** -133, 2.0 ** -126)])
def test_smallest_scale(amax, scale):
    assert ref.smallest_scale(amax) == scale


def test_appending_token_by_token_or_at_once_gives_the_same_scale():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((16, 2, 64)) * 2.0 ** rng.integers(-6, 6, (16, 1, 1))
    x = inputs.bits_to_f64(inputs.to_bits(x.astype(np.float32), inputs.BF16), inputs.BF16)
    codes, scale = np.zeros((3, 2, 16, 64), np.uint8), np.ones((3, 2), np.float32)
    at_once = ref.append(x, np.arange(16, 32), codes, scale, 16)
    for t in range(16):
        codes, scale = ref.append(x[t:t + 1], [16 + t], codes, scale, 16)
    assert np.array_equal(scale, at_once[1])
    # re-encoding by powers of two rounds only what falls below the normal range: half of 2^-9 per growth
    a, b = inputs.e4m3_bits_to_f64(codes), inputs.e4m3_bits_to_f64(at_once[0])
    assert np.max(np.abs(a - b)) <= 2.0 ** -9
