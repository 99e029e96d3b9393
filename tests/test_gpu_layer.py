"""The operators around the attention run together as a model runs them: one pre-norm transformer layer,
forward and backward, against the same layer in 64 bits."""
import math

import pytest
import torch
import torch.autograd.forward_ad as fwAD

DEV = "cuda:0"


def _weights(D, H, Hkv, d, F, dtype, g):
    def normal(*shape):
        return torch.randn(shape, generator=g)
    return {"n1w": 1 + 0.2 * normal(D), "n1b": 0.2 * normal(D), "n2w": 1 + 0.2 * normal(D), "n2b": 0.2 * normal(D),
            "qkv": (normal((H + 2 * Hkv) * d, D) * D ** -0.5).to(dtype), "o": (normal(D, H * d) * (H * d) ** -0.5).to(dtype),
            "gate_up": (normal(2 * F, D) * D ** -0.5).to(dtype), "down": (normal(D, F) * F ** -0.5).to(dtype)}


def _layer(x, w, pos, freqs, cu, H, Hkv, d, prefix, cp_P):
    """One layer by this package's operators (the projections between them are torch's)."""
    from vlm_zigzag_head_gb300.autograd import cp_attention, gated_ffn, layer_norm, rope
    T, F = x.shape[0], w["down"].shape[1]
    qkv = (layer_norm(x, w["n1w"], w["n1b"]) @ w["qkv"].t()).view(T, H + 2 * Hkv, d)
    q, k = rope(qkv[:, :H], qkv[:, H:H + Hkv], pos, inv_freq=freqs, amplitude=1.1)
    out, _ = cp_attention(q, k, qkv[:, H + Hkv:].contiguous(), cu, cp_P, prefix)
    x = x + out.reshape(T, H * d) @ w["o"].t()
    return x + gated_ffn(layer_norm(x, w["n2w"], w["n2b"]), w["gate_up"][:F], w["gate_up"][F:], w["down"],
                         activation="gelu_tanh")


def _layer64(x, w, pos, freqs, cu, H, Hkv, d):
    """The same from the definitions, in the tensors' precision (64 bits)."""
    def norm(v, a, b):
        c = v - v.mean(-1, keepdim=True)
        return c / (c.square().mean(-1, keepdim=True) + 1e-5).sqrt() * a + b
    T, F = x.shape[0], w["down"].shape[1]
    qkv = (norm(x, w["n1w"], w["n1b"]) @ w["qkv"].t()).view(T, H + 2 * Hkv, d)
    t = pos.double()[:, None] * torch.tensor(freqs, dtype=torch.float64)
    c, s = 1.1 * t.cos()[:, None], 1.1 * t.sin()[:, None]
    a, b = qkv[:, :H + Hkv, :d // 2], qkv[:, :H + Hkv, d // 2:]
    qk = torch.cat([a * c - b * s, b * c + a * s], -1)
    k, v = (z.repeat_interleave(H // Hkv, 1) for z in (qk[:, H:], qkv[:, H + Hkv:]))
    seen = torch.zeros(T, T, dtype=torch.bool)
    for i, j in zip(cu, cu[1:]):
        seen[i:j, i:j] = torch.ones(j - i, j - i).tril().bool()
    p = torch.einsum("ihd,jhd->hij", qk[:, :H], k) * d ** -0.5
    p = p.masked_fill(~seen, -math.inf).softmax(-1)
    x = x + torch.einsum("hij,jhd->ihd", p, v).reshape(T, H * d) @ w["o"].t()
    h = norm(x, w["n2w"], w["n2b"]) @ w["gate_up"].t()
    g = h[:, :F]
    act = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    return x + (act * h[:, F:]) @ w["down"].t()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_layer_forward_and_backward(dtype):
    """fp32: every operator holds 1e-5, and the layer chains about ten of them, forward and backward:
    1e-4.  bf16: the layer rounds about ten activations to bf16 on its way, each by 2^-8 / sqrt(3) of
    random sign (1.7e-3 on average, as measured on one operator), forward and again backward:
    sqrt(20) 1.7e-3 = 8e-3, twice that allowed."""
    import vlm_zigzag_head_gb300 as cp
    g = torch.Generator().manual_seed(0)
    H, Hkv, d, D, F, prefix = 4, 2, 64, 192, 352, 9
    cu = [0, prefix + 64, 2 * prefix + 64 + 32]
    T = cu[-1]
    w = _weights(D, H, Hkv, d, F, dtype, g)
    x, dy = torch.randn(T, D, generator=g).to(dtype), torch.randn(T, D, generator=g).to(dtype)
    pos = torch.cat([torch.arange(b - a) for a, b in zip(cu, cu[1:])]).to(torch.int32) + 3000
    freqs = cp.rope_frequencies(d, scaling="by_parts", factor=4.0, trained_length=1024)

    ref = {k: v.double().requires_grad_(True) for k, v in {**w, "x": x}.items()}
    want = _layer64(ref["x"], ref, pos, freqs, cu, H, Hkv, d)
    want_grads = torch.autograd.grad(want, list(ref.values()), dy.double())

    dev = {k: v.to(DEV).requires_grad_(True) for k, v in {**w, "x": x}.items()}
    got = _layer(dev["x"], dev, pos.to(DEV), freqs, cu, H, Hkv, d, prefix, 2)
    grads = torch.autograd.grad(got, list(dev.values()), dy.to(DEV))
    tol = 1e-4 if dtype == torch.float32 else 1.6e-2
    for name, a, b in zip(["y", *ref], [got, *grads], [want, *want_grads]):
        a, b = a.detach().double().cpu(), b.detach()
        assert a.shape == b.shape and torch.isfinite(a).all()
        assert float((a - b).norm() / b.norm()) <= tol, (name, float((a - b).norm() / b.norm()))


@pytest.mark.gpu
def test_a_captured_decoding_step():
    """The forms for single tokens, captured once and replayed on new inputs: norm, rotation in place
    and feed-forward block give the bits of plain calls."""
    import vlm_zigzag_head_gb300 as cp
    g = torch.Generator().manual_seed(1)
    H, Hkv, d, D, F = 8, 2, 64, 256, 640
    w = {k: v.to(DEV) for k, v in _weights(D, H, Hkv, d, F, torch.bfloat16, g).items()}
    x = torch.zeros(3, D, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(3, dtype=torch.int32, device=DEV)

    def step():
        n = cp.cp_layer_norm_fwd(x, w["n1w"], w["n1b"])[0]
        qkv = (n @ w["qkv"].t()).view(3, H + 2 * Hkv, d)
        cp.cp_rope_fwd(qkv[:, :H], qkv[:, H:H + Hkv], pos, inplace=True)
        return qkv, cp.cp_gated_ffn_fwd(n, w["gate_up"][:F], w["gate_up"][F:], w["down"])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        x.copy_(torch.randn(3, D, generator=g).to(torch.bfloat16))
        pos.copy_(torch.tensor([5 * i, 70000 + i, 1], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)


class _NoGradient(torch.autograd.Function):
    """Passes its input on; backward has nothing to say about it."""

    @staticmethod
    def forward(ctx, x):
        return x.clone()

    @staticmethod
    def backward(ctx, g):
        return None


@pytest.mark.gpu
def test_outputs_without_a_gradient_and_forward_mode():
    from vlm_zigzag_head_gb300.autograd import gated_ffn, layer_norm, rope
    x = torch.randn(5, 64, device=DEV)
    w, wd = torch.randn(128, 64, device=DEV), torch.randn(64, 128, device=DEV)
    q, pos = torch.randn(5, 2, 64, device=DEV), torch.arange(5, dtype=torch.int32, device=DEV)
    calls = (lambda t: layer_norm(t), lambda t: gated_ffn(t, w, w, wd),
             lambda t: rope(t.view(5, 1, 64), q, pos)[0])
    for call in calls:
        leaf = x.clone().requires_grad_(True)
        grad, = torch.autograd.grad(_NoGradient.apply(call(leaf)).sum() + leaf.sum(), leaf)
        assert torch.equal(grad, torch.ones_like(grad))
        with fwAD.dual_level(), pytest.raises(NotImplementedError):
            call(fwAD.make_dual(x, x))


@pytest.mark.gpu
def test_in_place_rotation_of_a_saved_tensor_is_noticed():
    import vlm_zigzag_head_gb300 as cp
    q = torch.randn(4, 2, 64, device=DEV, requires_grad=True)
    pos = torch.arange(4, dtype=torch.int32, device=DEV)
    h = q * 1.0
    y = (h * h).sum()       # saves h
    cp.cp_rope_fwd(h.detach(), torch.randn(4, 1, 64, device=DEV), pos, inplace=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    z = torch.randn(4, 3, 64, device=DEV)
    for bad in ((z[:, :2], z[:, 1:]), (z[:, :1].expand(4, 2, 64), z[:, 2:])):
        with pytest.raises(cp.CpError):
            cp.cp_rope_fwd(*bad, pos, inplace=True)


@pytest.mark.gpu
def test_waits_that_run_out_for_a_batch_of_rows():
    import vlm_zigzag_head_gb300 as cp
    g = torch.Generator().manual_seed(2)
    x, wg, wd = (torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV) for s in ((40, 1024), (2048, 1024), (512, 2048)))
    ws, seen = cp.Workspace(), []
    y = cp.cp_gated_ffn_fwd(x, wg, wg, wd)
    cp.cp_set_wait_limit(1)
    try:
        for _ in range(3):
            cp.cp_gated_ffn_fwd(x, wg, wg, wd, workspace=ws)
            seen.append(cp.cp_workspace_status(ws))
    finally:
        cp.cp_set_wait_limit(0)
    assert all(s in (0, 7) for s in seen) and 7 in seen, seen
    assert torch.equal(cp.cp_gated_ffn_fwd(x, wg, wg, wd, workspace=ws), y) and cp.cp_workspace_status(ws) == 0


@pytest.mark.gpu
def test_bounds_checked_build_agrees():
    """The checked library runs the feed-forward products without an index out of range, to the same bits."""
    import vlm_zigzag_head_gb300 as cp
    from vlm_zigzag_head_gb300 import build
    build.build(checked=True)
    g = torch.Generator().manual_seed(3)
    for T in (1, 40, 300):
        x, wg, wd, dy = (torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)
                         for s in ((T, 264), (520, 264), (136, 520), (T, 136)))

        def run():
            ws = cp.Workspace()
            y, gate, up = cp.cp_gated_ffn_fwd(x, wg, wg, wd, keep=True, workspace=ws)
            first = cp.cp_workspace_status(ws)
            out = cp.cp_gated_ffn_bwd(x, wg, wg, wd, gate, up, dy, workspace=ws)
            assert first == 0 and cp.cp_workspace_status(ws) == 0
            return (y, *out)
        want = run()
        with cp._binding.bounds_checked():
            got = run()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
