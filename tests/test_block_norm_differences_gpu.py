"""The block norm's fp32 gradients against differences of its own forward, along random directions."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn

from test_block_norm_gpu import EPS, FULL, formulas, make

pytestmark = pytest.mark.gpu
NAMES = dict(x="dx", gate="dgate", residual="dresidual", w_post="dw_post", res_scale="dres_scale", w_pre="dw_pre")


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("width", [64, 300, 1032, 37])
def test_random_directions(width, sigmoid):
    """Central differences of sum h dh + sum y dy, each element moved by a quarter either way. What a difference
    of that step is off the derivative (by the second order) comes from the float64 formulas at the same points;
    what is left is rounding: of the two values, 64 roundings of 2^-24 of the terms' magnitudes each, and of the
    gradient, 2^-16 of its terms' as in its own test."""
    flags = gdn.GDN_FLAG_GATE_SIGMOID if sigmoid else 0
    p, dh, dy = make((6, 2, width), "f32", FULL, seed=width)
    d = {k: v.cuda() for k, v in p.items()}
    _, _, stats = gdn.gdn_block_norm_fwd(d["x"], **{k: v for k, v in d.items() if k != "x"}, eps=EPS, flags=flags)
    grads = gdn.gdn_block_norm_bwd(d["x"], stats, dh.cuda(), dy.cuda(), **{k: v for k, v in d.items() if k != "x"},
                                   eps=EPS, flags=flags)
    exact, gmag = formulas(p, dh, dy, sigmoid), formulas(p, dh, dy, sigmoid, size=True)
    g = torch.Generator().manual_seed(1)

    def kernel(q):
        q = {k: v.cuda() for k, v in q.items()}
        h, y, _ = gdn.gdn_block_norm_fwd(q["x"], **{k: v for k, v in q.items() if k != "x"}, eps=EPS, flags=flags)
        return float((h.double().cpu() * dh.double()).sum() + (y.double().cpu() * dy.double()).sum())

    def formula(q, size=False):
        o = formulas(q, sigmoid=sigmoid, size=size)
        a, b = (dh.double().abs(), dy.double().abs()) if size else (dh.double(), dy.double())
        return float((o["h"] * a).sum() + (o["y"] * b).sum())

    for k, name in NAMES.items():
        for _ in range(3):
            v = torch.randint(0, 2, p[k].shape, generator=g) * 2.0 - 1.0
            lo, hi = {**p, k: p[k] - 0.25 * v}, {**p, k: p[k] + 0.25 * v}
            moved = hi[k].double() - lo[k].double()
            higher = formula(hi) - formula(lo) - float((exact[name] * moved).sum())
            got = kernel(hi) - kernel(lo) - higher
            want = float((grads[name].double().cpu() * moved).sum())
            tol = 2.0 ** -18 * (formula(hi, size=True) + formula(lo, size=True)) + 2.0 ** -16 * float((gmag[name] * moved.abs()).sum())
            assert abs(got - want) <= tol, (name, got, want, tol)
            # along a random direction the terms of a sum over n elements leave about its square root: the bound
            # is far below what the direction sees
            assert tol <= 0.05 * float((exact[name] * moved).norm()), (name, tol)
