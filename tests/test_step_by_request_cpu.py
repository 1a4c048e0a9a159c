"""Refusals of fa_paged_update_by_request without a GPU."""
import pytest

from exact_io_aware_30_gb300 import build, fa

FAKE = 0x7F0000001000  # never dereferenced: validation fails first
GB = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return fa.load()


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), fa.FA_ERR_INVALID_ARG), (dict(rows=-1), fa.FA_ERR_INVALID_ARG), (dict(B=0), fa.FA_ERR_INVALID_ARG),
    (dict(B=1 << 16, rows=1 << 15), fa.FA_ERR_INVALID_ARG), (dict(bs=48), fa.FA_ERR_UNSUPPORTED),
    (dict(slots=None), fa.FA_ERR_INVALID_ARG), (dict(positions=FAKE + 8 * GB + 2), fa.FA_ERR_MISALIGNED),
    # four requests of eight rows: 128 bytes of slots
    (dict(positions=FAKE + 7 * GB + 124), fa.FA_ERR_INVALID_ARG), (dict(state_out=FAKE), fa.FA_ERR_INVALID_ARG)])
def test_refused(kw, status):
    names = ("seq_lens", "delta", "table", "ring", "state", "lens_out", "state_out", "slots", "positions", "status")
    a = {n: FAKE + i * GB for i, n in enumerate(names)}
    a.update(B=4, max_blocks=8, ring_size=64, bs=16, rows=8)
    a.update(kw)
    assert fa.load().fa_paged_update_by_request(*[a[n] for n in names], a["B"], a["max_blocks"], a["ring_size"], a["bs"],
                                                a["rows"], None) == status
