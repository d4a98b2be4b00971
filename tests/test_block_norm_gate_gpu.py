"""The gate of fp32 rows to fp32's own accuracy, in every form of the kernels."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn

pytestmark = pytest.mark.gpu

# Relative errors, u = 2^-24 one rounding: exp(-g) within 1 ulp is 2u, 1 + exp another u, the reciprocal within
# 1 ulp 2u, so s is within 5u; h = x g s takes two products more. exp(-g) s is within 2 + 5 + 1 u, its product
# with s 5 + 1 more, and dh x d two products more.
U = 2.0 ** -24
ACT, SLOPE = (5 + 2) * U, (8 + 6 + 2) * U


@pytest.mark.parametrize("width", [64, 128, 101, 640, 1001, 2056, 4096])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_fp32_gate(width, sigmoid):
    g = torch.Generator().manual_seed(width)
    shape = (64, 1, width)
    x, dh = ((torch.rand(*shape, generator=g) + 0.5) * (torch.randint(0, 2, shape, generator=g) * 2 - 1) for _ in range(2))
    gate = torch.rand(*shape, generator=g) * 80 - 40
    flags = gdn.GDN_FLAG_GATE_SIGMOID if sigmoid else 0
    h, _, stats = gdn.gdn_block_norm_fwd(x.cuda(), gate=gate.cuda(), flags=flags)
    grads = gdn.gdn_block_norm_bwd(x.cuda(), stats, dh.cuda(), gate=gate.cuda(), flags=flags)
    x, dh, gate = x.double(), dh.double(), gate.double()
    s, rest = torch.sigmoid(gate), torch.sigmoid(-gate)
    act = s if sigmoid else gate * s

    def close(got, ref, rel):
        err = ((got.double().cpu() - ref).abs() / (rel * ref.abs() + 1e-300)).max()
        assert float(err) <= 1, float(err)

    close(h, x * act, ACT)
    close(grads["dx"], dh * act, ACT)
    if sigmoid:  # (silu's slope is a sum that cancels near g = -1.28)
        close(grads["dgate"], dh * x * s * rest, SLOPE)


@pytest.mark.parametrize("width", [520, 3080, 6152])
def test_fp32_gate_among_all_parts(width):
    """Residual zero and scale one: y beside h, whose gate has the same accuracy after two norms."""
    g = torch.Generator().manual_seed(width)
    shape = (16, 1, width)
    x = (torch.rand(*shape, generator=g) + 0.5) * (torch.randint(0, 2, shape, generator=g) * 2 - 1)
    gate, zero = torch.rand(*shape, generator=g) * 80 - 40, torch.zeros(shape)
    one = torch.ones(width).cuda()
    h, _, _ = gdn.gdn_block_norm_fwd(x.cuda(), gate=gate.cuda(), residual=zero.cuda(), w_pre=one)
    ref = x.double() * gate.double() * torch.sigmoid(gate.double())
    err = ((h.double().cpu() - ref).abs() / (ACT * ref.abs() + 1e-300)).max()
    assert float(err) <= 1, float(err)
