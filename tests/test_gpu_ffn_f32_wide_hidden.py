"""fp32 calls of up to 64 rows whose hidden layer is wide enough to fill the GPU with single tiles: sums
that are not shared out, products of many tiles, rows that end inside a tile.  Against 64 bits on the
same GPU, with the method's fp32 tolerance."""
import pytest
import torch

from gpu_util import F32_REL

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("T,D,F,D_out,act", [(33, 136, 40000, 72, "silu"), (64, 64, 20480, 64, "gelu"),
                                             (25, 1032, 19464, 8, "silu"), (3, 2048, 6144, 2048, "gelu_tanh")])
def test_matches_64_bits(T, D, F, D_out, act):
    import vlm_zigzag_head_gb300 as cp
    g = torch.Generator(device=DEV).manual_seed(T)

    def normal(*s):
        return torch.randn(s, generator=g, device=DEV)
    x, wg, wu, wd, dy = normal(T, D), normal(F, D) * D ** -0.5, normal(F, D) * D ** -0.5, \
        normal(D_out, F) * F ** -0.5, normal(T, D_out)
    ws = cp.Workspace()
    y, gate, up = cp.cp_gated_ffn_fwd(x, wg, wu, wd, act, keep=True, workspace=ws)
    got = [y, *cp.cp_gated_ffn_bwd(x, wg, wu, wd, gate, up, dy, act, workspace=ws)]
    assert cp.cp_workspace_status(ws) == 0
    leaves = [t.double().requires_grad_(True) for t in (x, wg, wu, wd)]
    a = leaves[0] @ leaves[1].t()
    a = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[act](a)
    want = (a * (leaves[0] @ leaves[2].t())) @ leaves[3].t()
    want = [want.detach(), *torch.autograd.grad(want, leaves, dy.double())]
    for name, p, q in zip(("y", "dx", "dw_gate", "dw_up", "dw_down"), got, want):
        assert float((p.double() - q).norm() / q.norm()) <= F32_REL, name
