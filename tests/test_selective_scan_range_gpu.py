"""Selective scan where a chunk's decay leaves float32's range while the states do not, and where A is -infinity."""
import math

import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn
from tests.mixer_reference import UNIT, scan_seq, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bound", [None, 1])  # chunks, and token by token (forward)
@pytest.mark.parametrize("T,D", [(4000, 32), (2000, 2048)])  # chunks carried eight at a time, and one by one
@pytest.mark.parametrize("sign", [1, -1])
def test_states_grow_and_decay_beyond_the_factors_range(sign, T, D, bound):
    """Eight tokens within a chunk change the state by 10^39, or 10^-39; the others leave it as it is."""
    gen = torch.Generator(device="cuda").manual_seed(T + D)
    S, at, rate = 16, 96, 89.8 / 8
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    dims, seqs = gdn.binding.GdnScanDims(D, 1, S, gdn.GDN_F32, 0), gdn.binding.GdnPacked(T, 1, 1, 1 << 20, None, None)
    assert gdn.load().gdn_selective_scan_workspace_bytes(dims, seqs, T) > 0  # it is split
    u, dt = torch.zeros(T, D, device="cuda"), torch.zeros(T, D, device="cuda")
    dt[at:at + 8] = 1.0
    A = torch.full((D, S), sign * rate, device="cuda")
    B = C = torch.ones(T, 1, S, device="cuda")
    h0, dh = ((1 + torch.rand(1, D, S, generator=gen, device="cuda")) * 10.0 ** (-20 * sign) for _ in range(2))
    y, h, kept = gdn.gdn_selective_scan_fwd(u, dt, A, B, C, h0=h0, cu_seqlens=cu, max_q=bound, save=bound is None)
    factor = torch.exp(A.double() * 8)
    # eight factors of exponents up to rate each, or one of their sum: the error of a step is UNIT (1 + 4 |exponent|)
    off = 9 * UNIT * (1 + 4 * rate)
    want = h0.double() * factor
    within("h", h, want, off * want)
    ref = torch.cat((h0.double().sum(-1).expand(at, D), want.sum(-1).expand(T - at, D)))
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[at:at + 8] = False
    within("y", y[keep], ref[keep], off * ref[keep])
    if bound is not None:
        return
    g = gdn.gdn_selective_scan_bwd(u, dt, A, B, C, torch.zeros_like(y), kept, dh_final=dh, need_dh0=True, cu_seqlens=cu)
    want = dh.double() * factor
    within("dh0", g["dh0"], want, off * want)
    want = (8 * dh.double() * h0.double() * factor)[0]  # G a h_{t-1} is the same for all eight
    within("dA", g["dA"], want, 3 * off * want)
    ddt = (sign * rate * dh.double() * h0.double() * factor)[0].sum(-1)
    within("ddt", g["ddt"][at:at + 8], ddt.expand(8, D), 3 * off * ddt.abs())


@pytest.mark.parametrize("bound", [None, 1])
@pytest.mark.parametrize("T", [1, 13, 1605])
def test_a_rate_of_minus_infinity_forgets_at_once(T, bound):
    gen = torch.Generator(device="cuda").manual_seed(T)
    D, S = 24, 16
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    u, dy = (torch.randn(T, D, generator=gen, device="cuda") for _ in range(2))
    dt = 1 + torch.rand(T, D, generator=gen, device="cuda")
    A = -torch.rand(D, S, generator=gen, device="cuda")
    A[3:, 2:5] = -200.0  # e^-200 is zero too
    B, C = (torch.randn(T, 1, S, generator=gen, device="cuda") for _ in range(2))
    h0, dh = (torch.randn(1, D, S, generator=gen, device="cuda") for _ in range(2))
    ref = scan_seq(u, dt, A, B, C, softplus=False, h0=h0[0], dy=dy, dh=dh[0])
    A[3:, 2:5] = -math.inf
    y, h, kept = gdn.gdn_selective_scan_fwd(u, dt, A, B, C, h0=h0, cu_seqlens=cu, max_q=bound, save=bound is None)
    within("y", y, *ref["y"])
    within("h", h[0], *ref["h"])
    if bound is None:
        g = gdn.gdn_selective_scan_bwd(u, dt, A, B, C, dy, kept, dh_final=dh, need_dh0=True, cu_seqlens=cu)
        within("du", g["du"], *ref["du"])
        within("dh0", g["dh0"][0], *ref["dh0"])
        within("dA", g["dA"], *ref["dA"])
        within("ddt", g["ddt"], *ref["ddt"])
