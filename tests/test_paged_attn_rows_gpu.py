"""gdn_paged_attn with queries of very different sizes in one call: every row within the bound of its own scores."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn

from paged_reference import UNIT, Paged, attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,length", [([1] * 6, [7, 40, 900, 16, 333, 2000]), ([4, 9], [700, 2500]), ([150, 70], [150, 800])])
def test_rows_within_their_own_bounds(dtype, new, length):
    """The bounds of attention_bounds with each row's own largest sum |q k| scale in place of the call's."""
    scale = 128 ** -0.5
    c = Paged(new, length, 8, 2, 128, 64, dtype, seed=29)
    q = c.normal(c.N, 8, 128)
    small = torch.tensor([2.0 ** -(i % 7) for i in range(c.N)])[:, None, None] * torch.tensor([1.0, 0.25] * 4)[None, :, None]
    q = (q.float() * 4 * small).to(c.dt)
    kc, vc, table, cu, lens = c.cuda()
    lse = torch.empty(c.N, 8, device="cuda")
    out = gdn.gdn_paged_attn(q.cuda(), kc, vc, table, cu, lens, scale, max_q=max(new), max_kv=max(length), lse=lse)
    ref, mag, rlse, _ = attention(c, q, scale)
    size, keys = torch.zeros(c.N, 8, dtype=torch.float64), torch.zeros(c.N, 1, dtype=torch.float64)
    for tok, b, pos in c.tokens():
        K = c.dense(c.kc, b)[:, :pos + 1].abs().repeat_interleave(4, 0)
        size[tok] = (torch.einsum("hd,hkd->hk", q[tok].double().abs(), K) * scale).amax(-1)
        keys[tok] = pos + 1
    fp32 = 2.0 ** -18 * (1 + size) + keys * 2.0 ** -24
    tol = mag * fp32[..., None] + ref.abs() * UNIT[dtype] + (mag * UNIT["bf16"] if dtype == "bf16" else 0) + 1e-30
    err = (out.double().cpu() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    ltol = 2.0 ** -19 * (1 + size) + rlse.abs() * 2.0 ** -21 + keys * 2.0 ** -24
    assert bool(((lse.double().cpu() - rlse).abs() <= ltol).all())
