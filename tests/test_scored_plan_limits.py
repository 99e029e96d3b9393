"""Score plans at the ends of what their sizes can hold (host only)."""
import ctypes

import numpy as np
import pytest

from vlm_zigzag_head_gb300 import _binding as B

I32 = ctypes.POINTER(ctypes.c_int32)


def _size(cu, heads, sms):
    return B.lib().cp_score_plan_size(cu.ctypes.data_as(I32), len(cu) - 1, None, 0, heads, sms, None, 0)


@pytest.mark.parametrize("short", [0, 4000, 5000])
def test_units_near_the_largest_32_bit_number(cplib, short):
    """Samples of one token give one unit each and head: the list of units and of the 4096 blocks' shares
    has more entries than 32 bits count, and still takes four bytes for each of them."""
    heads = 127
    n = (2 ** 31 - 1 - short) // heads
    cu = np.arange(n + 1, dtype=np.int32)
    size = _size(cu, heads, 4096)
    # units and the blocks' shares; per sample two items of 128 bytes, a run and a tile of 32
    least = 4 * (n * heads + 4096 + 1) + n * (128 + 128 + 32 + 32)
    assert least < size < least + 4096


def test_more_units_than_32_bits_hold(cplib):
    n = (2 ** 31 - 1) // 127 + 1
    assert _size(np.arange(n + 1, dtype=np.int32), 127, 152) == 0
    assert b"too many work units" in B.lib().cp_last_error()
