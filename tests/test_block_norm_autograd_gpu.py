"""block_norm under autograd."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn

from test_block_norm_gpu import EPS, FULL, make

pytestmark = pytest.mark.gpu


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
