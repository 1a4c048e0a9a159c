"""Attention over the 8-bit paged cache with V scales of very different sizes
beside each other."""
import pytest

torch = pytest.importorskip("torch")

import decode_formula as formula
from exact_io_aware_30_gb300 import fa

pytestmark = pytest.mark.gpu

ROWS = [(1, 1), (4, 1), (8, 1), (4, 4), (4, 6), (8, 4), (20, 2)]  # H / Hkv, Sq


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from exact_io_aware_30_gb300 import build
    build.build()
    fa.load()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    assert fa.device_error() == fa.FA_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G,Sq", ROWS)
def test_a_large_scale_where_there_is_no_weight(G, Sq, d, dtype):
    # one block's V scale is 2^e times the others', and its keys' weights are 2^-e to 2^-(e + 30) of theirs: all or
    # most of O comes from the small scales (fp16: e up to 12, so that O fits)
    lens = [40, 300, 120, 900]
    for e in (6, 12, 14, 20, 40, 90):
        p = formula.problem(4, 2 * G, 2, Sq, d, 16, lens, dtype, seed=e)
        q, kc, vc, ks, vs, table, _ = p
        q[..., 0] = 8.0
        vs.copy_(torch.where(vs.isnan(), vs, vs * 2.0 ** -6))
        for b, L in enumerate(lens):
            block = int(table[b, L // 16 // 2])
            kc[block, :, :, 0] = 0xFE  # -448
            kc[block, :, :, 1:] = 0
            ks[block] = (e + 15 * (b % 3)) * 0.6931 / (8 * 448)
            vs[block] = 2.0 ** (e - 14)
        got = fa.decode_paged_fp8(*p, 900, scale=1.0)
        formula.check(got, *p, 1.0, "none")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("G,Sq,d", [(2, 4, 128), (1, 3, 64), (4, 5, 256), (8, 4, 128)])
def test_a_large_scale_that_only_the_last_row_sees(G, Sq, d, dtype):
    # a draft's last token begins a block and is an outlier: the rows in front of it do not see it
    L = 16 * 20 + 1
    p = formula.problem(2, 2 * G, 2, Sq, d, 16, [L, L], dtype, seed=Sq)
    q, kc, vc, ks, vs, table, _ = p
    for b in range(2):
        vs[int(table[b, 20])] = 2.0 ** (3 if dtype == torch.float16 else 40)
        vs[table[b, :20].long()] *= 2.0 ** -10
    got = fa.decode_paged_fp8(*p, L, mask="causal")
    formula.check(got, *p, d ** -0.5, "causal")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("G,Sq", ROWS)
def test_zero_scales_and_scales_at_the_ends_of_the_range(G, Sq, dtype):
    # an empty block's scale (2^-126) and zeros beside ordinary ones; scales that are all tiny; negative ones
    lens = [100, 260]
    for kind in range(3):
        p = formula.problem(2, 2 * G, 2, Sq, 128, 16, lens, dtype, seed=kind)
        vs = p[4]
        for b in range(2):
            if kind == 0:
                vs[int(p[5][b, 1])], vs[int(p[5][b, 3])] = 2.0 ** -126, 0.0
            elif kind == 1:
                vs[p[5][b].clamp(min=0).long()] = 2.0 ** -110
            else:
                vs[int(p[5][b, 2])] *= -2.0 ** 13
        got = fa.decode_paged_fp8(*p, 260)
        formula.check(got, *p, 128 ** -0.5, "none")
