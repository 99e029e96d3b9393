"""The autograd functions of the operators beside the attention at the edges of what autograd asks: outputs
without a gradient."""
import pytest
import torch

DEV = "cuda:0"


class _NoGradient(torch.autograd.Function):
    """Passes its input on; backward has nothing to say about it."""

    @staticmethod
    def forward(ctx, x):
        return x.clone()

    @staticmethod
    def backward(ctx, g):
        return None


def _scored_inputs(dtype=torch.bfloat16, device=DEV):
    g = torch.Generator().manual_seed(1)
    return [torch.randn((90, h, 64), generator=g).to(dtype).to(device) for h in (2, 1, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scored_attention_whose_output_gets_no_gradient(dtype):
    """The engine still runs the node; the inputs then get what their other uses give."""
    from vlm_zigzag_head_gb300 import ScorePlan
    from vlm_zigzag_head_gb300.autograd import cp_attention_scored
    plan = ScorePlan([0, 90], 2, rel_buckets=[0, 1], device=DEV)
    leaves = [x.requires_grad_(True) for x in _scored_inputs(dtype)]
    bias = torch.randn(2, 2, device=DEV).requires_grad_(True)
    out, _ = cp_attention_scored(*leaves, plan, rel_bias=bias)
    loss = _NoGradient.apply(out).float().sum() + leaves[2].float().sum()
    dq, dk, dv, db = torch.autograd.grad(loss, leaves + [bias], allow_unused=True)
    assert dq is None and dk is None and db is None
    assert torch.equal(dv, torch.ones_like(dv))


@pytest.mark.gpu
def test_norm_rope_whose_outputs_get_no_gradient():
    from vlm_zigzag_head_gb300.autograd import qk_norm_rope
    q, k, _ = (x.requires_grad_(True) for x in _scored_inputs())
    pos = torch.arange(90, dtype=torch.int32, device=DEV)
    w = torch.ones(64, device=DEV, requires_grad=True)
    qn, kn = qk_norm_rope(q, k, pos, w, w)
    dq, dk, dw = torch.autograd.grad(_NoGradient.apply(qn).float().sum() + kn.float().sum(), (q, k, w))
    assert not dq.any() and dk.any() and dw.any()
