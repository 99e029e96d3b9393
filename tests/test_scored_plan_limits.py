"""Score plans at the ends of what their sizes can hold (host only)."""
import ctypes
import subprocess
import sys

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


CHILD = """
import ctypes, resource, sys
lib = ctypes.CDLL(sys.argv[1])
lib.cp_score_plan_size.restype = ctypes.c_size_t
lib.cp_last_error.restype = ctypes.c_char_p
def size():
    cu = (ctypes.c_int32 * 2)(0, 2 ** 31 - 1)
    return lib.cp_score_plan_size(cu, 1, None, 0, 1, 152, None, 0)
if sys.argv[2] == "free":
    assert size() > 0
else:   # no room for the lists of tiles by length (16 million entries)
    with open("/proc/self/statm") as f:
        used = int(f.read().split()[0]) * resource.getpagesize()
    soft, hard = resource.getrlimit(resource.RLIMIT_AS)
    resource.setrlimit(resource.RLIMIT_AS, (used + (32 << 20), hard))
    assert size() == 0 and lib.cp_last_error()
    resource.setrlimit(resource.RLIMIT_AS, (soft, hard))
    assert size() > 0
"""


@pytest.mark.parametrize("memory", ["free", "short"])
def test_no_exception_leaves_the_size_query(cplib, memory):
    """Out of memory is an error like any other: 0 and a message."""
    r = subprocess.run([sys.executable, "-c", CHILD, B.lib_path(), memory], capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0, (r.returncode, r.stderr[-1000:])
