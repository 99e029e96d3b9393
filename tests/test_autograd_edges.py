"""The autograd functions of the operators beside the attention at the edges of what autograd asks: outputs
without a gradient, and forward-mode derivatives, which they have none of."""
import pytest
import torch
import torch.autograd.forward_ad as fwAD

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


def _duals(*tensors):
    """The same tensors, each in turn as a dual one."""
    for i, x in enumerate(tensors):
        yield [fwAD.make_dual(t, torch.ones_like(t)) if j == i else t for j, t in enumerate(tensors)]


@pytest.mark.parametrize("grad", [False, True])
def test_dual_tensors_go_through_the_autograd_function(grad):
    """...which has no forward-mode rule and says so; a plain call would drop the tangent."""
    from vlm_zigzag_head_gb300.autograd import _wants_grad
    x, y = torch.ones(3), torch.ones(3)
    with torch.set_grad_enabled(grad):
        assert not _wants_grad(x, None, y)
        with fwAD.dual_level():
            assert not _wants_grad(x, None, y)
            for a in _duals(x, y):
                assert _wants_grad(a[0], None, a[1])
        torch.func.jvp(lambda t: (t, _seen.append(_wants_grad(t, None)))[0], (x,), (y,))
    assert _seen.pop() is True


_seen = []


@pytest.mark.gpu
@pytest.mark.parametrize("grad", [False, True])
def test_forward_mode_is_refused(grad):
    from vlm_zigzag_head_gb300 import ScorePlan
    from vlm_zigzag_head_gb300.autograd import cp_attention, cp_attention_scored, qk_norm_rope
    plan = ScorePlan([0, 90], 2, rel_buckets=[0, 1], device=DEV)
    q, k, v = _scored_inputs()
    pos, w = torch.arange(90, dtype=torch.int32, device=DEV), torch.ones(64, device=DEV)
    bias, slopes = torch.zeros(2, 2, device=DEV), torch.ones(2, device=DEV)
    with torch.set_grad_enabled(grad), fwAD.dual_level():
        for a in _duals(q, k, v, bias):
            with pytest.raises(NotImplementedError):
                cp_attention_scored(*a[:3], plan, rel_bias=a[3])
        with pytest.raises(NotImplementedError):
            cp_attention_scored(q, k, v, plan, slopes=fwAD.make_dual(slopes, slopes))
        for a in _duals(q, k, w):
            with pytest.raises(NotImplementedError):
                qk_norm_rope(a[0], a[1], pos, a[2], None)
        with pytest.raises(NotImplementedError):     # as the unmodified attention
            cp_attention(fwAD.make_dual(q, q), k, v, [0, 90], 1)
