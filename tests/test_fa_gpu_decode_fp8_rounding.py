"""Attention over the 8-bit paged cache where rounding shows: weights that nearly
cancel, and query rows with components far below their largest."""
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
def test_two_keys_that_nearly_cancel(G, Sq, d, dtype):
    # V is 1 for the one and -1 for the other: O = tanh(x / 2) of their scores' difference x, small beside
    # the weights, so that a weight's rounding is not hidden by O's
    B = 40
    p = formula.problem(B, 2 * G, 2, Sq, d, 16, [2] * B, dtype, seed=G)
    q, kc, vc, ks, vs, table, lens = p
    q.zero_()
    q[..., 0] = (1.0 + torch.arange(B, device="cuda").view(B, 1, 1) / 32).to(dtype)
    kc.zero_()
    for b in range(B):
        block = int(table[b, 0])
        kc[block, :, 0, 0] = 0x38
        vc[block, :, 0], vc[block, :, 1] = 0x38, 0xB8
    ks.fill_(2.0 ** -6)
    vs.fill_(1.0)
    got = fa.decode_paged_fp8(*p, 2, scale=1.0)
    formula.check(got, *p, 1.0, "none")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("G,Sq", ROWS)
def test_components_far_below_their_row_s_largest(G, Sq, dtype):
    # 129/128 2^-14 and less beside a component of 1, against keys that read only those
    p = formula.problem(2, 2 * G, 2, Sq, 64, 16, [200, 60], dtype, seed=5)
    q, kc, vc, ks, vs, table, _ = p
    g = torch.Generator(device="cuda").manual_seed(6)
    size = torch.exp2(-torch.randint(8, 20, q.shape, device="cuda", generator=g).float())
    q.copy_((q.float() * size).to(dtype))
    q[..., 1] = 129 / 128 * 2.0 ** -14
    q[..., 0] = 1.0
    kc[..., 0] = 0
    got = fa.decode_paged_fp8(*p, 200, scale=200.0)
    formula.check(got, *p, 200.0, "none")
