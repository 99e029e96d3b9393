"""A rotation in place writes past autograd: where a gradient or a tangent would go through it, the
call is refused; detached tensors and no_grad leave the graph, and the bits are those of the copy."""
import pytest
import torch
import torch.autograd.forward_ad as fwAD

from vlm_zigzag_head_gb300 import CpError, cp_rope_bwd, cp_rope_fwd

REFUSED = "being differentiated: not in place"


def _graph_tensors(device):
    leaf = torch.randn(4, 2, 64, device=device, requires_grad=True)
    return leaf, leaf * 1.0, (leaf * 1.0)[:, :1]


@pytest.mark.parametrize("call", [cp_rope_fwd, cp_rope_bwd])
def test_refused_before_anything_is_touched(call):
    """No GPU: the refusal comes before any other check."""
    pos, plain = torch.arange(4, dtype=torch.int32), torch.randn(4, 1, 64)
    for x in _graph_tensors("cpu"):
        for q, k in ((x, plain), (plain, x)):
            before = x.detach().clone()
            with pytest.raises(CpError, match=REFUSED):
                call(q, k, pos, inplace=True)
            assert torch.equal(x, before) and x._version == 0
        with torch.no_grad(), pytest.raises(CpError, match="CUDA device"):   # the next check
            call(x, plain, pos, inplace=True)
    with fwAD.dual_level(), pytest.raises(CpError, match=REFUSED):
        call(fwAD.make_dual(plain, plain), plain, pos, inplace=True)


@pytest.mark.gpu
@pytest.mark.parametrize("call", [cp_rope_fwd, cp_rope_bwd])
def test_refused_or_outside_the_graph(call):
    dev = "cuda:0"
    pos = torch.arange(4, dtype=torch.int32, device=dev) + 7
    for x in _graph_tensors(dev):
        k = torch.randn(4, 1, 64, device=dev)
        want = call(x.detach(), k, pos)
        for a, b in ((x, k.clone()), (k.clone(), x)):
            before = x.detach().clone()
            with pytest.raises(CpError, match=REFUSED):
                call(a, b, pos, inplace=True)
            assert torch.equal(x, before)
        free = x.detach().clone()
        got = call(free, k.clone(), pos, inplace=True)
        assert got[0] is free and all(torch.equal(a, b) for a, b in zip(got, want))
        with torch.no_grad():
            got = call(x, k.clone(), pos, inplace=True)
        assert got[0] is x and all(torch.equal(a, b) for a, b in zip(got, want))
