"""The 4-bit append into caches past 4 GB: the codes and words of K and of V, whose rows differ, each in its place."""
import numpy as np
import pytest

import int4_reference as ref
from exact_io_aware_30_gb300 import fa

torch = pytest.importorskip("torch")

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


def test_append_past_32_bits_writes_both_caches_codes_and_words():
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    bs, Hkv, d, group = 128, 8, 256, 32
    blocks = (1 << 32) // (bs * Hkv * d // 2) + 4  # codes past 2^32 bytes
    cache = [torch.full((blocks, Hkv, bs, n), fill, dtype=dt, device="cuda")
             for n, fill, dt in ((d // 2, 0xA5, torch.uint8), (d // 2, 0x5A, torch.uint8),
                                 (d // group, 0x3F804500, torch.int32), (d // group, 0x40004600, torch.int32))]
    rng = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(4, Hkv, d, device="cuda", generator=rng).bfloat16() for _ in range(2))
    at = [blocks - 2, blocks - 1, 0]
    before = [t[at].cpu().numpy() for t in cache]
    slots = torch.tensor([(blocks - 1) * bs + 7, (blocks - 2) * bs + 1, -1, 5], dtype=torch.int32, device="cuda")
    fa.cache_append_int4(k, v, slots, *cache)
    for i, x in ((0, k), (1, v)):
        codes, words = ref.append(x.double().cpu().numpy(), np.array([bs + 7, 1, -1, 2 * bs + 5]), before[i], before[i + 2], bs, group)
        assert np.array_equal(cache[i][at].cpu().numpy(), codes)
        assert np.array_equal(cache[i + 2][at].cpu().numpy(), words)
    # nothing else has changed
    for i, fill in enumerate((0xA5, 0x5A, 0x3F804500, 0x40004600)):
        rest = cache[i][1:blocks - 2]
        assert all(bool((rest[j:j + 4096] == fill).all()) for j in range(0, len(rest), 4096))
