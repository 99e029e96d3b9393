"""How the feed-forward block's products are cut into units, for calls without rows (host only).

The functions are C++ ones of the library, called in a process of their own: a division by zero ends a
process on some machines (x86), where on others (Arm) it gives 0."""
import subprocess
import sys

import pytest

from vlm_zigzag_head_gb300 import _binding as B

CHILD = """
import ctypes, sys
lib = ctypes.CDLL(sys.argv[1])

class Cut(ctypes.Structure):      # GemmCut
    _fields_ = [("tiles", ctypes.c_int64), ("k_tiles", ctypes.c_int), ("whole", ctypes.c_int64),
                ("shares", ctypes.c_int)]

class Cost(ctypes.Structure):     # GemmCost
    _fields_ = [("tile_n", ctypes.c_int), ("step", ctypes.c_double), ("epilogue", ctypes.c_double),
                ("least_k", ctypes.c_int)]

cut = getattr(lib, "_ZN6cpattn12cut_productsEPNS_7GemmCutEiiRKNS_8GemmCostE")
cut.restype = ctypes.c_double
cut.argtypes = [ctypes.POINTER(Cut), ctypes.c_int, ctypes.c_int, ctypes.POINTER(Cost)]
share = getattr(lib, "_ZN6cpattn9share_f32Ellliii")
share.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 3

def products(*shapes):
    p = (Cut * 3)()
    for c, (tiles, k_tiles) in zip(p, shapes):
        c.tiles, c.k_tiles = tiles, k_tiles
    time = cut(p, len(shapes), 76, ctypes.byref(Cost(256, 0.29, 2.0, 4)))
    return time, [(c.whole, c.shares) for c in p[:len(shapes)]]

if sys.argv[2] == "products":
    # no rows: a product of no tiles, and ones of tiles without k
    for shapes in ([(0, 16)], [(0, 32), (24, 0), (12, 0)], [(0, 0)]):
        time, cuts = products(*shapes)
        assert time >= 0 and cuts == [(tiles, 1) for tiles, _ in shapes], (shapes, time, cuts)
    # with rows they are cut as before: 8 tiles of 96 k tiles for 76 pairs of CTAs
    (whole, shares), = products((8, 96))[1]
    assert whole == 0 and shares > 1, (whole, shares)
else:
    for M, N, K, outputs, phases in ((0, 1360, 512, 1, 1), (0, 512, 1360, 1, 2), (1360, 512, 0, 2, 1),
                                     (512, 1360, 0, 1, 1), (0, 512, 0, 1, 1)):
        assert share(M, N, K, outputs, phases, 152) == 1, (M, N, K)
    assert share(64, 1360, 512, 1, 1, 152) > 1
"""


@pytest.mark.parametrize("what", ["products", "f32"])
def test_calls_without_rows_are_planned(cplib, what):
    r = subprocess.run([sys.executable, "-c", CHILD, B.lib_path(), what], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stderr[-1000:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [0, 1])
def test_workspace_sizes_without_rows(cplib, dtype):
    """Both sizes hold the status word, and no partial sums."""
    f = B.GatedFfnDesc()
    f.dtype = f.grad_dtype = dtype
    f.T, f.D, f.F, f.D_out = 0, 64, 128, 32
    f.w_gate_stride = f.w_up_stride = 64
    f.w_down_stride = 128
    sizes = cplib.cp_gated_ffn_fwd_workspace_size(f), cplib.cp_gated_ffn_bwd_workspace_size(f)
    f.T = 1
    one = cplib.cp_gated_ffn_fwd_workspace_size(f), cplib.cp_gated_ffn_bwd_workspace_size(f)
    assert all(0 < a < b for a, b in zip(sizes, one)), (sizes, one)
