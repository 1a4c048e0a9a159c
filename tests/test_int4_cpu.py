"""Refusals of the 4-bit paged cache's entry points, without a GPU (every call here
fails validation before it touches the device), and the reference's own format."""
import ctypes

import numpy as np
import pytest

import int4_reference as ref
from exact_io_aware_30_gb300 import build, fa, inputs

FAKE = 0x7F0000001000  # 256-byte aligned, never dereferenced: validation fails first
GB = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return fa.load()


# ------------------------------------------------------------------ append

def _append(**kw):
    a = dict(k=FAKE, v=FAKE + GB, kt=1024, kh=128, vt=1024, vh=128, slots=FAKE + 2 * GB, kc=FAKE + 3 * GB,
             vc=FAKE + 4 * GB, ks=FAKE + 5 * GB, vs=FAKE + 6 * GB, T=4, Hkv=8, d=128, group=32, bs=16, blocks=64,
             dtype=fa.DTYPE_BF16)
    a.update(kw)
    return fa.load().fa_cache_append_int4(a["k"], a["v"], a["kt"], a["kh"], a["vt"], a["vh"], a["slots"], a["kc"],
                                          a["vc"], a["ks"], a["vs"], a["T"], a["Hkv"], a["d"], a["group"], a["bs"],
                                          a["blocks"], a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=fa.DTYPE_FP32), fa.FA_ERR_UNSUPPORTED), (dict(d=96), fa.FA_ERR_UNSUPPORTED),
    (dict(group=16), fa.FA_ERR_UNSUPPORTED), (dict(group=128), fa.FA_ERR_UNSUPPORTED), (dict(group=0), fa.FA_ERR_UNSUPPORTED),
    (dict(bs=24), fa.FA_ERR_UNSUPPORTED), (dict(Hkv=0), fa.FA_ERR_INVALID_ARG), (dict(T=-1), fa.FA_ERR_INVALID_ARG),
    (dict(T=(1 << 30) + 1), fa.FA_ERR_INVALID_ARG), (dict(blocks=0), fa.FA_ERR_INVALID_ARG),
    (dict(blocks=1 << 27), fa.FA_ERR_INVALID_ARG), (dict(Hkv=65536), fa.FA_ERR_INVALID_ARG),
    (dict(v=None), fa.FA_ERR_INVALID_ARG), (dict(slots=None), fa.FA_ERR_INVALID_ARG), (dict(kt=-1), fa.FA_ERR_INVALID_ARG),
    (dict(vh=(1 << 40) + 1), fa.FA_ERR_INVALID_ARG), (dict(kt=1 << 40, T=1 << 20), fa.FA_ERR_INVALID_ARG),
    (dict(k=FAKE + 1), fa.FA_ERR_MISALIGNED), (dict(kc=FAKE + 3 * GB + 8), fa.FA_ERR_MISALIGNED),
    (dict(vs=FAKE + 6 * GB + 4), fa.FA_ERR_MISALIGNED), (dict(slots=FAKE + 2 * GB + 2), fa.FA_ERR_MISALIGNED),
    (dict(kc=FAKE), fa.FA_ERR_INVALID_ARG), (dict(vc=FAKE + 3 * GB + 4096), fa.FA_ERR_INVALID_ARG),
    (dict(ks=FAKE + 3 * GB + 64), fa.FA_ERR_INVALID_ARG), (dict(vs=FAKE + 5 * GB), fa.FA_ERR_INVALID_ARG),
    (dict(ks=FAKE + 2 * GB), fa.FA_ERR_INVALID_ARG)])
def test_append_refused(kw, status):
    assert _append(**kw) == status


def test_append_of_no_rows_is_ok():
    assert _append(T=0, k=None, v=None, slots=None) == fa.FA_OK


# ------------------------------------------------------------------ reading back

def _read(**kw):
    a = dict(kc=FAKE, vc=FAKE + GB, ks=FAKE + 2 * GB, vs=FAKE + 3 * GB, table=FAKE + 4 * GB, lens=FAKE + 5 * GB,
             starts=FAKE + 6 * GB, k=FAKE + 7 * GB, kst=(2 * 40 * 128, 40 * 128, 128), v=FAKE + 8 * GB,
             vst=(2 * 40 * 128, 40 * 128, 128), B=3, Hkv=2, rows=40, d=128, group=32, bs=16, max_blocks=4, blocks=64,
             dtype=fa.DTYPE_BF16)
    a.update(kw)
    arr = lambda s: None if s is None else (ctypes.c_longlong * 3)(*s)
    return fa.load().fa_cache_read_int4(a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["lens"], a["starts"], a["k"],
                                        arr(a["kst"]), a["v"], arr(a["vst"]), a["B"], a["Hkv"], a["rows"], a["d"],
                                        a["group"], a["bs"], a["max_blocks"], a["blocks"], a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=fa.DTYPE_FP32), fa.FA_ERR_UNSUPPORTED), (dict(d=32), fa.FA_ERR_UNSUPPORTED),
    (dict(group=48), fa.FA_ERR_UNSUPPORTED), (dict(bs=8), fa.FA_ERR_UNSUPPORTED), (dict(B=0), fa.FA_ERR_INVALID_ARG),
    (dict(rows=-1), fa.FA_ERR_INVALID_ARG), (dict(B=1, rows=(1 << 30) + 1), fa.FA_ERR_INVALID_ARG),
    (dict(Hkv=65536), fa.FA_ERR_INVALID_ARG), (dict(max_blocks=0), fa.FA_ERR_INVALID_ARG),
    (dict(max_blocks=1 << 28), fa.FA_ERR_INVALID_ARG), (dict(B=1 << 20, rows=1 << 12), fa.FA_ERR_INVALID_ARG),
    (dict(kc=None), fa.FA_ERR_INVALID_ARG), (dict(lens=None), fa.FA_ERR_INVALID_ARG), (dict(v=None), fa.FA_ERR_INVALID_ARG),
    (dict(kst=None), fa.FA_ERR_INVALID_ARG), (dict(vst=(10240, 5120, -128)), fa.FA_ERR_INVALID_ARG),
    (dict(kst=(10240, 5120, 127)), fa.FA_ERR_INVALID_ARG), (dict(kst=(0, 5120, 128)), fa.FA_ERR_INVALID_ARG),
    (dict(kst=(1 << 41, 5120, 128)), fa.FA_ERR_INVALID_ARG), (dict(k=FAKE + 7 * GB + 1), fa.FA_ERR_MISALIGNED),
    (dict(ks=FAKE + 2 * GB + 8), fa.FA_ERR_MISALIGNED), (dict(starts=FAKE + 6 * GB + 2), fa.FA_ERR_MISALIGNED),
    (dict(v=FAKE + 7 * GB + 256), fa.FA_ERR_INVALID_ARG), (dict(k=FAKE), fa.FA_ERR_INVALID_ARG),
    (dict(v=FAKE + 4 * GB), fa.FA_ERR_INVALID_ARG), (dict(v=FAKE + 6 * GB), fa.FA_ERR_INVALID_ARG)])
def test_read_refused(kw, status):
    assert _read(**kw) == status


def test_read_of_no_rows_is_ok():
    assert _read(rows=0, k=None, v=None) == fa.FA_OK


# ------------------------------------------------------------------ decode

def _decode(**kw):
    a = dict(q=FAKE, kc=FAKE + GB, vc=FAKE + 2 * GB, ks=FAKE + 3 * GB, vs=FAKE + 4 * GB, table=FAKE + 5 * GB,
             lens=FAKE + 6 * GB, o=FAKE + 7 * GB, lse=FAKE + 8 * GB, ws=FAKE + 9 * GB, ws_bytes=GB, B=2, H=8, Hkv=2,
             Sq=1, d=128, group=32, bs=16, max_blocks=8, blocks=64, max_len=128, scale=0.1, mask=fa.MASK_CAUSAL,
             dtype=fa.DTYPE_BF16)
    a.update(kw)
    return fa.load().fa_decode_paged_int4(
        a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["lens"], a["o"], a["lse"], a["ws"], a["ws_bytes"],
        a["B"], a["H"], a["Hkv"], a["Sq"], a["d"], a["group"], a["bs"], a["max_blocks"], a["blocks"], a["max_len"],
        a["scale"], a["mask"], a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=fa.DTYPE_FP32), fa.FA_ERR_UNSUPPORTED), (dict(d=80), fa.FA_ERR_UNSUPPORTED),
    (dict(group=128), fa.FA_ERR_UNSUPPORTED), (dict(group=-32), fa.FA_ERR_UNSUPPORTED),
    (dict(bs=256), fa.FA_ERR_UNSUPPORTED), (dict(mask=fa.MASK_SLIDING_WINDOW), fa.FA_ERR_UNSUPPORTED),
    (dict(H=9), fa.FA_ERR_INVALID_ARG), (dict(Hkv=0), fa.FA_ERR_INVALID_ARG), (dict(Sq=0), fa.FA_ERR_INVALID_ARG),
    (dict(Sq=33), fa.FA_ERR_UNSUPPORTED), (dict(max_len=0), fa.FA_ERR_INVALID_ARG), (dict(max_len=129), fa.FA_ERR_INVALID_ARG),
    (dict(B=1, max_blocks=1 << 27, max_len=0x7fffffff - 511), fa.FA_ERR_INVALID_ARG), (dict(blocks=0), fa.FA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), fa.FA_ERR_INVALID_ARG), (dict(scale=-0.1), fa.FA_ERR_INVALID_ARG),
    (dict(ks=None), fa.FA_ERR_INVALID_ARG), (dict(kc=FAKE + GB + 8), fa.FA_ERR_MISALIGNED),
    (dict(vs=FAKE + 4 * GB + 4), fa.FA_ERR_MISALIGNED), (dict(ws=FAKE + 9 * GB + 16), fa.FA_ERR_MISALIGNED),
    (dict(q=FAKE + 8), fa.FA_ERR_MISALIGNED), (dict(lse=FAKE + 8 * GB + 2), fa.FA_ERR_MISALIGNED)])
def test_decode_refused(kw, status):
    assert _decode(**kw) == status


def test_decode_workspace_query_needs_a_place_for_its_answer():
    assert fa.load().fa_decode_int4_workspace_query(2, 8, 2, 1, 128, 32, 16, 8, 64, 128, 0, 0, None) == fa.FA_ERR_INVALID_ARG
    assert fa.decode_int4_workspace_query(2, 8, 2, 1, 96, 32, 16, 8, 64, 128) == (fa.FA_ERR_UNSUPPORTED, 0)
    assert fa.decode_int4_workspace_query(2, 8, 2, 1, 128, 16, 16, 8, 64, 128) == (fa.FA_ERR_UNSUPPORTED, 0)


@pytest.mark.parametrize("kw", [dict(d=96), dict(group=16), dict(block_size=8)])
def test_an_empty_cache_of_sizes_that_are_not_held_is_refused(kw):
    a = dict(num_blocks=2, H_kv=1, block_size=16, d=64, group=32, device="cpu")
    a.update(kw)
    with pytest.raises(fa.FAError):
        fa.int4_cache(**a)


# ------------------------------------------------------------------ the reference itself

def test_words_and_codes_there_and_back():
    s, z = np.array([[0.25, 1.0078125]], np.float32), np.array([[7.0, -2048.0]])
    assert np.array_equal(ref.unpack_words(ref.words(s, z)), (s.astype(np.float64), z))
    c = np.arange(64) % 16
    v = ref.values(ref.pack(c), ref.words(s, z)[0])
    assert np.array_equal(v, np.concatenate([0.25 * (c[:32] - 7.0), 1.0078125 * (c[32:] + 2048.0)]))


@pytest.mark.parametrize("dtype", [inputs.BF16, inputs.FP16])
def test_a_quantised_value_is_within_half_a_step(dtype):
    rng = np.random.default_rng(1)
    for shift in (0.0, 5.0, -300.0):
        x = inputs.bits_to_f64(inputs.to_bits((rng.standard_normal(64) + shift).astype(np.float32), dtype), dtype)
        c, s, z = ref.quantise(x, 32)
        assert c.min() >= 0 and c.max() <= 15 and np.abs(z).max() <= 2048
        v = ref.values(ref.pack(c), ref.words(s, z))
        assert np.all(np.abs(v - x) <= np.repeat(s, 32).astype(np.float64) / 2)
        # the step is the range over 15, or 2^-11 of the largest, rounded up by at most 2^-7
        wide = np.array([max(np.ptp(g) / 15, np.abs(g).max() / 2048) for g in x.reshape(2, 32)])
        assert np.all(s >= wide * (1 - 2.0 ** -23)) and np.all(s <= wide * (1 + 2.0 ** -7))
