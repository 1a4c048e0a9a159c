"""Attention over the 4-bit paged cache on whole grids where one warp of each CTA gives up waiting: the others wind
down from wherever they are, without waiting for tiles that nobody began to copy."""
import time

import pytest

import test_fa_gpu_int4 as base
from exact_io_aware_30_gb300 import fa, inputs

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from exact_io_aware_30_gb300 import build
    build.build()
    fa.load()
    torch.cuda.set_device(0)
    yield


@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("B,H,Hkv,d,group", [(40, 16, 16, 64, 32), (40, 16, 16, 128, 32), (40, 128, 16, 128, 64), (20, 512, 16, 128, 32),
                                             (20, 320, 16, 256, 32), (20, 16, 16, 256, 64)])
def test_a_warp_that_gives_up_stops_its_cta_soon(B, H, Hkv, d, group, bs):
    lens = [1500 - 37 * i for i in range(B)]
    p = base._problem(B, H, Hkv, 1, d, group, bs, lens, inputs.BF16, seed=bs + d)
    dev = base._device(p)
    want = fa.decode_paged_int4(*dev, 1500)
    torch.cuda.synchronize()
    assert fa.device_error() == fa.FA_OK
    fa.set_debug_stall_ms(20)
    try:
        began = time.time()
        fa.decode_paged_int4(*dev, 1500)
        torch.cuda.synchronize()
        took = time.time() - began
    finally:
        fa.set_debug_stall_ms(0)
    assert fa.device_error() == fa.FA_ERR_DEVICE_TIMEOUT
    assert fa.device_error() == fa.FA_OK
    assert took < 1.0, took  # (a tile that is waited for in vain takes 2 s)
    o, lse = fa.decode_paged_int4(*dev, 1500)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
