"""gdn_paged_attn with a CTA per item over more sequences than a warp has lanes: empty sequences, rows without
keys, and the report of a length beyond the page table."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn

from paged_reference import Paged, attention, attention_bounds

pytestmark = pytest.mark.gpu


def _many(first=50):
    """75 sequences, some without new tokens, some whose first tokens or all tokens stand before position 0."""
    new = [first] + [0 if b % 5 == 0 else 40 + b * 13 % 60 for b in range(1, 75)]
    length = [n + 37 * b % 300 if n else b for b, n in enumerate(new)]
    for b in range(3, 75, 7):
        length[b] = max(new[b] - 10, 0)
    for b in range(9, 75, 11):
        length[b] = 0
    c = Paged(new, length, 24, 24, 64, 16, "bf16", seed=31)
    assert c.N // 256 * 24 >= 304  # two full items per SM: a CTA per item
    return c, c.normal(c.N, 24, 64, std=1.5)


def test_many_sequences_with_a_cta_per_item():
    c, q = _many()
    kc, vc, table, cu, lens = c.cuda()
    out = torch.full(q.shape, float("nan"), dtype=c.dt, device="cuda")
    lse = torch.full((c.N, 24), float("nan"), dtype=torch.float32, device="cuda")
    gdn.gdn_paged_attn(q.cuda(), kc, vc, table, cu, lens, 0.125, max_q=max(c.new), max_kv=max(c.length), out=out, lse=lse)
    out, lse = out.double().cpu(), lse.double().cpu()
    ref, mag, rlse, size = attention(c, q, 0.125)
    tol, ltol = attention_bounds(c, ref, mag, rlse, size)
    assert bool(((out - ref).abs() <= tol).all()), float(((out - ref).abs() / tol).max())
    none = torch.isinf(rlse)
    assert int(none.sum()) > 0 and bool((lse[none] == -float("inf")).all()) and bool((out[none] == 0).all())
    assert bool(((lse - rlse).abs()[~none] <= ltol.expand_as(rlse)[~none]).all())
    assert gdn.gdn_check_device_error() == 0


@pytest.mark.parametrize("first", [50, 0])
@pytest.mark.parametrize("b", [0, 20, 43, 74])
def test_a_length_beyond_the_table_is_reported_wherever_it_stands(first, b):
    """Sequence 0 with new tokens and without, and sequences of each group of 32."""
    c, q = _many(first)
    kc, vc, table, cu, lens = c.cuda()
    table[table < 0] = 0  # the clamped length reads every page of the row
    lens[b] = 100000
    assert gdn.gdn_check_device_error() == 0
    gdn.gdn_paged_attn(q.cuda(), kc, vc, table, cu, lens, 0.125, max_q=max(c.new), max_kv=max(c.length))
    assert gdn.gdn_check_device_error() == gdn.binding.GDN_ERR_INTERNAL
    assert gdn.gdn_check_device_error() == 0
