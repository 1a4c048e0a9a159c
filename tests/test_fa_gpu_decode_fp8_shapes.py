"""Attention over the 8-bit paged cache on grids that are full, so that a CTA walks
from unit to unit, its rings turn over and shares end inside units on odd tiles:
every number of rows per K/V head, with units cut and whole, against the formula."""
import pytest

torch = pytest.importorskip("torch")

import decode_formula as formula
from exact_io_aware_30_gb300 import fa

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


def _run(p, max_len, mask):
    got = fa.decode_paged_fp8(*p, max_len, mask=mask)
    formula.check(got, *p, p[0].shape[-1] ** -0.5, mask)
    return got


# H / Hkv and Sq: rows per K/V head of every kernel size (1, 2-4, 5-8, 9-16, 17-24, 25-32) and of several chunks
ROWS = [(1, 1), (1, 2), (4, 1), (3, 2), (4, 2), (3, 3), (16, 1), (4, 5), (6, 4), (7, 4), (32, 1), (8, 5), (26, 2), (128, 1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G,Sq", ROWS)
def test_units_cut_between_ctas_that_walk_many_tiles(G, Sq, d, dtype):
    # over 2,500 tiles, six and more for each CTA whatever the kernel's CTAs per SM, in units of 1 to 14
    lens = [1700, 129, 1, 0, 640, 1281, 300, 128, 999, 1536, 257, 40] * 5
    p = formula.problem(len(lens), 8 * G, 8, Sq, d, (16, 32, 64, 128)[(G + Sq) % 4], lens, dtype, seed=G * 10 + Sq)
    _run(p, 1700, "causal" if Sq > 1 else "none")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G,Sq", ROWS)
def test_whole_units_several_to_a_cta_and_the_same_data_cut(G, Sq, d, dtype):
    lens = [512, 1, 384, 129, 0, 257, 128, 100, 511, 385, 30, 256] * 10
    p = formula.problem(len(lens), 8 * G, 8, Sq, d, (32, 64, 128, 16)[(G + Sq) % 4], lens, dtype, seed=G * 20 + Sq,
                        max_blocks=64)
    mask = "causal" if Sq > 1 else "none"
    _run(p, 512, mask)
    _run(p, 1000, mask)  # a bound above four tiles: the same requests with their units cut


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G,Sq", [(1, 1), (4, 1), (2, 4), (4, 4), (4, 6), (8, 4)])
def test_one_long_request(G, Sq, d):
    # units of 71 tiles: each lies across several CTAs, and each CTA has several of its tiles
    p = formula.problem(1, 40 * G, 40, Sq, d, 64, [9001], torch.bfloat16, seed=d + G)
    _run(p, 9001, "causal")


def test_an_outlier_before_a_long_even_tail_within_one_cta():
    # 64 heads of 20,000 keys: a CTA has about 30 tiles of a unit.  A spike of weight 1 with V = 0, then
    # 2^-20 each: taken relative to the spike, the tail (2 % of the row) would be below the parts' steps
    H, d, bs, n = 64, 64, 128, 20000
    p = formula.problem(1, H, H, 1, d, bs, [n], torch.bfloat16, seed=3)
    q, kc, vc, ks, vs, table, lens = p
    q.zero_()
    q[..., 0] = 1.0
    kc.zero_()
    ks.fill_(1.0)
    vs.fill_(1.0)
    vc.fill_(0x38)  # 1.0
    first = int(table[0, 0])
    kc[first, :, 3, 0] = torch.tensor([14.0]).to(torch.float8_e4m3fn).view(torch.uint8).item()
    vc[first, :, 3] = 0
    got = fa.decode_paged_fp8(*p, n, scale=1.0)
    formula.check(got, *p, 1.0, "none")
    assert bool((got[0] > 0.01).all())
