"""Without a norm after the block, x does not enter dx: a non-finite x leaves the gradients of its row finite
but for those that multiply by it."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn

from paged_reference import UNIT
from test_block_norm_gpu import EPS, formulas, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [64, 128, 256, 101, 640, 1001, 2056, 4096, 6144])
@pytest.mark.parametrize("on", [("gate",), (), ("gate", "residual", "scale")])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_dx_without_a_norm_does_not_read_x(dtype, width, on, bad):
    p, dh, _ = make((5, 2, width), dtype, {k: k in on for k in ("post", "gate", "residual", "scale", "pre")}, seed=width)
    ref, mag = formulas(p, dh), formulas(p, dh, size=True)
    x = p["x"].clone()
    at = [(0, 0, 0), (2, 1, width // 2), (4, 1, width - 1)]
    for i in at:
        x[i] = bad
    d = {k: (None if v is None else v.cuda()) for k, v in p.items() if k != "x"}
    _, _, stats = gdn.gdn_block_norm_fwd(x.cuda(), **d, eps=EPS)
    g = gdn.gdn_block_norm_bwd(x.cuda(), stats, dh.cuda(), **d, eps=EPS)
    # one rounding to the type, and a chain of a few fp32 products, as for any dx
    tol = UNIT[dtype] * ref["dx"].abs() + 2.0 ** -16 * mag["dx"] + 1e-30
    assert bool(((g["dx"].double().cpu() - ref["dx"]).abs() <= tol).all())
    if "gate" in on:
        wrong = ~torch.isfinite(g["dgate"].cpu())
        assert int(wrong.sum()) == len(at) and all(bool(wrong[i]) for i in at)
