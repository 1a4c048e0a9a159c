"""The quantising append (fa_cache_append_fp8) with few live rows in a large padded
slot map, as a captured step with room for many tokens has it."""
import numpy as np
import pytest

import step_reference as ref
from exact_io_aware_30_gb300 import fa, inputs

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from exact_io_aware_30_gb300 import build
    build.build()
    fa.load()
    torch.cuda.set_device(0)


def _fresh(rng, blocks, Hkv, bs, d):
    codes = rng.integers(0, 256, (2, blocks, Hkv, bs, d)).astype(np.uint8)
    scale = (2.0 ** rng.integers(-9, 3, (2, blocks, Hkv))).astype(np.float32)
    return codes, scale


def _check(rng, slots, blocks, Hkv, bs, d):
    T = len(slots)
    x = torch.randn(T, Hkv, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(T)).bfloat16()
    codes, scale = _fresh(rng, blocks, Hkv, bs, d)
    t = [torch.from_numpy(c.copy()).cuda() for c in codes] + [torch.from_numpy(s.copy()).cuda() for s in scale]
    fa.cache_append_fp8(x, x, torch.from_numpy(slots.astype(np.int32)).cuda(), *t)
    live = np.flatnonzero(slots >= 0)
    rows = x[torch.from_numpy(live).cuda()].double().cpu().numpy()
    for i in range(2):
        want, want_scale = ref.append(rows, slots[live], codes[i], scale[i], bs)
        got = t[i].cpu().numpy()
        assert np.array_equal(t[2 + i].cpu().numpy(), want_scale)
        assert np.all((got == want) | (((got & 0x7F) == 0x7F) & ((want & 0x7F) == 0x7F)))


@pytest.mark.parametrize("T", [300, 700, 2500, 5000, 20000])
@pytest.mark.parametrize("where", ["front", "back", "middle", "far apart", "split block"])
def test_few_rows_among_many_skipped_ones(T, where):
    # one block's rows may have any number of skipped rows between them
    rng = np.random.default_rng(T)
    bs, Hkv, d, n = 16, 2, 64, 40
    blocks = 8
    chain = 5 + np.arange(n)
    live = rng.permutation(blocks)[chain // bs] * bs + chain % bs
    at = {"front": np.arange(n), "back": T - n + np.arange(n), "middle": T // 3 + np.arange(n),
          "far apart": np.sort(rng.permutation(T)[:n]),
          "split block": np.concatenate([np.arange(15), T - n + np.arange(15, n)])}[where]
    slots = np.full(T, -1)
    slots[at] = live
    _check(rng, slots, blocks, Hkv, bs, d)


def _time(call):
    for _ in range(3):
        call()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    best = float("inf")
    for _ in range(5):
        a.record()
        for _ in range(5):
            call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / 5)
    return best


@pytest.mark.parametrize("where", ["front", "far apart"])
def test_padding_costs_less_than_rows_would(where):
    # the same call with every row live moves 400 MB; 64 live rows move 0.4
    T, Hkv, d, bs = 65536, 8, 128, 16
    x = torch.randn(T, Hkv, d, device="cuda").bfloat16()
    kc, vc = (torch.zeros(T // bs, Hkv, bs, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(T // bs, Hkv, device="cuda") for _ in range(2))
    every = torch.arange(T, dtype=torch.int32, device="cuda")
    few = torch.full_like(every, -1)
    rows = torch.arange(64, device="cuda") * (1 if where == "front" else 1000)
    few[rows] = (torch.arange(64, device="cuda") * 7 * bs + 3).int()  # a block each, as in a decode step
    dense = _time(lambda: fa.cache_append_fp8(x, x, every, kc, vc, ks, vs))
    padded = _time(lambda: fa.cache_append_fp8(x, x, few, kc, vc, ks, vs))
    assert padded <= dense, (padded, dense)
