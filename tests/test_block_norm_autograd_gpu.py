"""block_norm under autograd: second derivatives are refused, outputs that a loss does not use, what is kept
for the backward."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn

from paged_reference import UNIT
from test_block_norm_gpu import EPS, FULL, formulas, make

pytestmark = pytest.mark.gpu
NAMES = dict(x="dx", gate="dgate", residual="dresidual", w_post="dw_post", res_scale="dres_scale", w_pre="dw_pre")


def _leaves(p):
    return {k: v.cuda().requires_grad_() for k, v in p.items() if v is not None}


def _call(d):
    return gdn.block_norm(d["x"], **{k: v for k, v in d.items() if k != "x"}, eps=EPS)


def test_second_derivatives_are_refused():
    """A gradient penalty: the second-order terms would be missing from the sum."""
    p, _, _ = make((6, 2, 128), "f32", FULL, seed=1)
    d = _leaves(p)
    h, y = _call(d)
    g, = torch.autograd.grad((h * y).sum(), d["x"], create_graph=True)
    with pytest.raises(RuntimeError):
        (y.sum() + g.square().sum()).backward()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [128, 640, 1001])
@pytest.mark.parametrize("use", ["h", "y"])
def test_a_loss_of_one_output(monkeypatch, dtype, width, use):
    """The gradient of the other output is none, not a tensor of zeros that is written and read; the weight
    behind it gets zeros."""
    p, dh, dy = make((9, 2, width), dtype, FULL, seed=2)
    seen, real = [], gdn.binding.gdn_block_norm_bwd
    monkeypatch.setattr(gdn.binding, "gdn_block_norm_bwd", lambda x, stats, dh, dy=None, **k: (seen.append((dh, dy)),
                                                                                              real(x, stats, dh, dy, **k))[1])
    d = _leaves(p)
    out = _call(d)[0 if use == "h" else 1]
    got = dict(zip(d, torch.autograd.grad(out, list(d.values()), (dh if use == "h" else dy).cuda())))
    (sdh, sdy), = seen
    assert (sdh is None) == (use == "y") and (sdy is None) == (use == "h")
    zero = torch.zeros_like(dh)
    args = (dh, zero) if use == "h" else (zero, dy)
    ref, mag = formulas(p, *args), formulas(p, *args, size=True)
    for k, g in got.items():
        r, m = ref[NAMES[k]], mag[NAMES[k]]
        assert bool(((g.double().cpu() - r).abs() <= UNIT[dtype] * r.abs() + 2.0 ** -16 * m + 1e-30).all()), k
    if use == "h":
        assert bool((got["w_pre"] == 0).all())


def test_neither_output_used_or_no_norm_before():
    p, dh, _ = make((9, 2, 128), "f32", dict(FULL, pre=False), seed=3)
    d = _leaves(p)
    h, y = _call(d)
    assert y is None
    got = torch.autograd.grad(h, list(d.values()), dh.cuda())
    ref = formulas(p, dh)
    for k, g in zip(d, got):
        assert float((g.double().cpu() - ref[NAMES[k]]).norm() / ref[NAMES[k]].norm()) <= 2.0 ** -16, k


@pytest.mark.parametrize("pre", [False, True])
def test_the_residual_is_kept_only_where_its_values_are_read(pre):
    """Without a norm before the next block the residual's gradient is dh itself."""
    p, dh, dy = make((4096, 1, 1024), "f32", dict(FULL, pre=pre), seed=4)
    d = _leaves(p)
    leaf = d.pop("residual")
    residual = leaf * 1.0
    size = residual.nbytes
    h, y = gdn.block_norm(d["x"], residual=residual, **{k: v for k, v in d.items() if k != "x"}, eps=EPS)
    before = torch.cuda.memory_allocated()
    del residual
    freed = before - torch.cuda.memory_allocated()
    assert freed == (0 if pre else size)
    outs, gs = ([h, y], [dh.cuda(), dy.cuda()]) if pre else ([h], [dh.cuda()])
    got = torch.autograd.grad(outs, [leaf, d["x"]], gs)
    ref, mag = formulas(p, dh, dy), formulas(p, dh, dy, size=True)
    for g, n in zip(got, ("dresidual", "dx")):
        assert bool(((g.double().cpu() - ref[n]).abs() <= UNIT["f32"] * ref[n].abs() + 2.0 ** -16 * mag[n] + 1e-30).all()), n
