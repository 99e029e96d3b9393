"""A training program can learn that a bounded device wait of the feed-forward block ran out: both
directions of the differentiable call use a workspace that is given, whose status says so."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_waits_that_run_out_in_training_are_reported(dtype):
    import vlm_zigzag_head_gb300 as cp
    from vlm_zigzag_head_gb300.autograd import gated_ffn
    g = torch.Generator().manual_seed(1)
    x, wg, wu, wd, dy = ((torch.randn(*s, generator=g) * s[1] ** -0.5).to(dtype).to(DEV)
                         for s in ((600, 512), (1024, 512), (1024, 512), (512, 1024), (600, 512)))
    leaves = [t.requires_grad_(True) for t in (x, wg, wu, wd)]
    want = gated_ffn(*leaves)
    grads = torch.autograd.grad(want, leaves, dy)
    ws, seen = cp.Workspace(), {"forward": [], "backward": []}
    for _ in range(3):
        cp.cp_set_wait_limit(1)
        try:
            gated_ffn(*leaves, workspace=ws)
            seen["forward"].append(cp.cp_workspace_status(ws))
        finally:
            cp.cp_set_wait_limit(0)
        y = gated_ffn(*leaves, workspace=ws)
        assert cp.cp_workspace_status(ws) == 0 and torch.equal(y, want)
        cp.cp_set_wait_limit(1)
        try:
            torch.autograd.grad(y, leaves, dy, retain_graph=True)
            seen["backward"].append(cp.cp_workspace_status(ws))
        finally:
            cp.cp_set_wait_limit(0)
        got = torch.autograd.grad(y, leaves, dy)
        assert cp.cp_workspace_status(ws) == 0 and all(torch.equal(a, b) for a, b in zip(got, grads))
    for way, s in seen.items():
        assert set(s) <= {0, 7} and 7 in s, (way, s)


def test_without_gradients_the_workspace_is_used_too():
    import vlm_zigzag_head_gb300 as cp
    from vlm_zigzag_head_gb300.autograd import gated_ffn
    x, w, wd = (torch.randn(*s, device=DEV) for s in ((40, 64), (128, 64), (64, 128)))
    ws = cp.Workspace()
    y = gated_ffn(x, w, w, wd, workspace=ws)
    assert ws.buf is not None and cp.cp_workspace_status(ws) == 0 and torch.equal(y, gated_ffn(x, w, w, wd))
