"""The autograd functions of the convolution and the scan as programs call them."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn

pytestmark = pytest.mark.gpu


def _model(gen, D, S):
    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    return [torch.nn.Parameter(t) for t in (-normal(D, S).abs() - 0.1, normal(D), normal(D) - 3)]  # A, D, dt_bias


def _inputs(gen, T, D, S, dtype=torch.bfloat16):
    return [torch.randn(1, T, *s, generator=gen, device="cuda").to(dtype) for s in ((D,), (D,), (1, S), (1, S))]


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_scan_without_gradients_keeps_nothing(mode):
    """Parameters that require gradients, gradients off: no states for a backward, and single tokens by their own kernel."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    D, S = 1024, 64
    A, skip, bias = _model(gen, D, S)
    u, dt, B, C = _inputs(gen, 4096, D, S)
    with mode():
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        y, h = gdn.selective_scan(u, dt, A, B, C, skip, None, bias, flags=gdn.GDN_FLAG_DT_SOFTPLUS)
        torch.cuda.synchronize()
        kept = 4096 // 8 * D * S * 4  # 134 MB
        assert torch.cuda.max_memory_allocated() - before < kept / 2
    want = gdn.gdn_selective_scan_fwd(u, dt, A.detach(), B, C, D=skip.detach(), dt_bias=bias.detach(), flags=gdn.GDN_FLAG_DT_SOFTPLUS)
    assert torch.equal(y, want[0]) and torch.equal(h, want[1]) and not y.requires_grad
    token = [t[:, :1].contiguous() for t in (u, dt, B, C)]
    gdn.gdn_profile_enable(True)
    gdn.gdn_profile_read()
    with mode():
        gdn.selective_scan(token[0], token[1], A, token[2], token[3], skip, None, bias, flags=gdn.GDN_FLAG_DT_SOFTPLUS)
    torch.cuda.synchronize()
    launches = {k: v[1] for k, v in gdn.gdn_profile_read().items() if v[1]}
    gdn.gdn_profile_enable(False)
    assert launches == {"selective_step_kernel": 1}
    # with gradients on they are kept, and go through
    y, _ = gdn.selective_scan(u, dt, A, B, C, skip, None, bias, flags=gdn.GDN_FLAG_DT_SOFTPLUS)
    assert y.requires_grad and bool(torch.isfinite(torch.autograd.grad(y.float().sum(), A)[0]).all())


def test_gradients_of_states_from_the_middle_of_a_tensor():
    """A loss over states concatenated with other values: their gradient begins at any element of a larger one."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    D, S = 20, 16
    A, skip, bias = _model(gen, D, S)
    u, dt, B, C = _inputs(gen, 9, D, S, torch.float32)
    w = torch.nn.Parameter(torch.randn(D, 4, generator=gen, device="cuda"))
    weights = torch.randn(1 + D * S, generator=gen, device="cuda")

    def grads(join):
        x, state = gdn.causal_conv(u, w)
        y, h = gdn.selective_scan(x, dt, A, B, C, skip, None, bias, flags=gdn.GDN_FLAG_DT_SOFTPLUS)
        if join:
            loss = (torch.cat((y.sum().view(1), h.reshape(-1))) * weights).sum()
            loss = loss + (torch.cat((y.sum().view(1), state.reshape(-1))) * weights[:1 + 3 * D]).sum()
        else:
            loss = y.sum() * weights[0] + (h.reshape(-1) * weights[1:]).sum()
            loss = loss + y.sum() * weights[0] + (state.reshape(-1) * weights[1:1 + 3 * D]).sum()
        return torch.autograd.grad(loss, (A, skip, bias, w))

    for a, b in zip(grads(True), grads(False)):
        assert torch.equal(a, b)
