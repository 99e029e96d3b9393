"""The feed-forward block on both sides of its tiles' ends, against the fp64 oracle.

The products of many rows have tiles of 256 rows, 256 or 128 columns (gate and up: half as many of each)
and steps of 64 k; fp32 beyond 64 rows 256 x 128.  bf16 forward calls of up to 8 and up to 128 rows and
fp32 ones of up to 24 and up to 64 have kernels of their own.  Bounds as in test_gpu_gated_ffn."""
import pytest
import torch

from test_gpu_gated_ffn import _check, _inputs

pytestmark = pytest.mark.gpu
WIDTHS = [(64, 128, 256), (72, 136, 264), (56, 120, 248), (128, 64, 128), (136, 264, 120)]   # D, F, D_out


@pytest.mark.parametrize("T", [255, 256, 257, 511, 512, 513, 769])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_around_a_tile(T, dtype):
    import vlm_zigzag_head_gb300 as cp
    for i, (D, F, D_out) in enumerate(WIDTHS):
        act = ("silu", "gelu", "gelu_tanh")[(T + i) % 3]
        x, wg, wu, wd, dy = _inputs(T, D, F, D_out, dtype, T + D)
        ws = cp.Workspace()
        y, gate, up = cp.cp_gated_ffn_fwd(x, wg, wu, wd, act, keep=True, workspace=ws)
        assert cp.cp_workspace_status(ws) == 0
        grads = cp.cp_gated_ffn_bwd(x, wg, wu, wd, gate, up, dy, act, workspace=ws)
        assert cp.cp_workspace_status(ws) == 0
        _check((y, *grads), x, wg, wu, wd, dy, act, dtype, torch.float32)


@pytest.mark.parametrize("dtype,edges", [(torch.bfloat16, (8, 9, 16, 17, 32, 33, 48, 49, 96, 97, 128, 129)),
                                         (torch.float32, (24, 25, 64, 65, 128, 129))])
def test_rows_where_the_kernels_change(dtype, edges):
    """The same rows, one more of them or not, to the last operand's rounding."""
    import vlm_zigzag_head_gb300 as cp
    x, wg, wu, wd, dy = _inputs(max(edges), 136, 264, 72, dtype, 5)
    for T in edges:
        ws = cp.Workspace()
        y, gate, up = cp.cp_gated_ffn_fwd(x[:T], wg, wu, wd, keep=True, workspace=ws)
        assert cp.cp_workspace_status(ws) == 0
        grads = cp.cp_gated_ffn_bwd(x[:T], wg, wu, wd, gate, up, dy[:T], workspace=ws)
        _check((y, *grads), x[:T], wg, wu, wd, dy[:T], "silu", dtype, torch.float32)
