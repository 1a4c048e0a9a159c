"""Plans of rotary positions whose frequencies are fewer or other than the call reads are
refused before anything is enqueued."""
import pytest

torch = pytest.importorskip("torch")

from exact_io_aware_30_gb300 import fa


@pytest.mark.parametrize("freq", [torch.zeros(31, dtype=torch.int64), torch.zeros(32), torch.zeros(32, dtype=torch.int32),
                                  torch.zeros(64, dtype=torch.int64)[::2]])
@pytest.mark.parametrize("call", [fa.rope, fa.rope_backward])
def test_a_plan_that_does_not_hold_its_frequencies_is_refused(call, freq):
    q = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(fa.FAError, match="frequencies") as e:
        call(q, None, fa.RopePlan(64, freq, 1.0))
    assert e.value.status == fa.FA_ERR_INVALID_ARG
