"""A single row has no stride: whatever a C caller's descriptor holds there, the call is that of a
contiguous row.  (A stride of 1 was taken for an operand whose rows lie side by side, by the fp32
backward on CUDA cores.)"""
import pytest
import torch

from vlm_zigzag_head_gb300 import _binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _call(dtype, x_stride, dy_stride, tensors, D, F, D_out):
    x, wg, wu, wd, dy = tensors
    f = B.GatedFfnDesc()
    f.dtype, f.grad_dtype, f.T, f.D, f.F, f.D_out = int(dtype == torch.bfloat16), 0, 1, D, F, D_out
    f.x_stride, f.dy_stride, f.w_gate_stride, f.w_up_stride, f.w_down_stride = x_stride, dy_stride, D, D, F
    L, stream = B.lib(), torch.cuda.current_stream().cuda_stream
    kept = [torch.empty(L.cp_gated_ffn_kept_size(f), dtype=torch.uint8, device=DEV) for _ in range(2)]
    sizes = L.cp_gated_ffn_fwd_workspace_size(f), L.cp_gated_ffn_bwd_workspace_size(f)
    ws = torch.empty(max(sizes), dtype=torch.uint8, device=DEV)
    y = torch.empty(D_out, dtype=dtype, device=DEV)
    grads = [torch.empty(D, dtype=dtype, device=DEV)] + \
        [torch.empty(s, device=DEV) for s in ((F, D), (F, D), (D_out, F))]
    at = [t.data_ptr() for t in (x, wg, wu, wd)]
    assert L.cp_gated_ffn_fwd(f, *at, y.data_ptr(), *(t.data_ptr() for t in kept), ws.data_ptr(), ws.numel(),
                              stream) == 0
    assert L.cp_gated_ffn_bwd(f, *at, *(t.data_ptr() for t in kept), dy.data_ptr(),
                              *(t.data_ptr() for t in grads), ws.data_ptr(), ws.numel(), stream) == 0
    torch.cuda.synchronize()
    return (y, *grads)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,F,D_out", [(64, 128, 40), (8, 8, 8), (520, 1360, 264)])
def test_any_stride_of_a_single_row(dtype, D, F, D_out):
    g = torch.Generator().manual_seed(D)
    tensors = [torch.randn(s, generator=g).to(dtype).to(DEV) for s in ((D,), (F, D), (F, D), (D_out, F), (D_out,))]
    want = _call(dtype, D, D_out, tensors, D, F, D_out)
    assert all(torch.isfinite(t).all() for t in want)
    for strides in ((1, D_out), (D, 1), (1, 1), (0, 0), (-3, 5), (1 << 40, -(1 << 40))):
        for a, b in zip(_call(dtype, *strides, tensors, D, F, D_out), want):
            assert torch.equal(a, b), strides
