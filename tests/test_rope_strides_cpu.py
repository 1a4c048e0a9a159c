"""Strides of fa_rope whose offsets would pass 63 bits are refused, without a GPU."""
import ctypes

import pytest

from exact_io_aware_30_gb300 import build, fa

FAKE = 0x7F0000001000  # never dereferenced: validation fails first
GB = 1 << 30


@pytest.mark.parametrize("stride", [(1 << 40) + 1, 1 << 61, (1 << 63) - 1])
def test_a_stride_of_the_positions_that_passes_the_limit_is_refused(stride):
    build.build()
    steps = (ctypes.c_longlong * 3)(4096, 128, 512)
    # (1 << 61: times 4 bytes and B - 1 = 8 the extent came round to a small number)
    assert fa.load().fa_rope(FAKE, steps, FAKE + GB, steps, FAKE + 2 * GB, steps, FAKE + 3 * GB, steps, FAKE + 5 * GB,
                             stride, 0, FAKE + 4 * GB, 1.0, 9, 4, 4, 8, 128, 128, 0, 0, fa.DTYPE_BF16,
                             None) == fa.FA_ERR_INVALID_ARG
