"""NaN in what a row sees reaches the row's output and its lse, and no other row's, in every schedule of
gdn_paged_attn: a NaN is not taken for a row without keys."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn

from paged_reference import Paged

pytestmark = pytest.mark.gpu
NAN = float("nan")

# new, length, Hq, Hk: the few-rows kernel with items held whole and cut between CTAs, and with bf16 the
# tcgen05 kernel by runs (items of one and of two row tiles, cut or not) and with a CTA per item
LAYOUTS = {
    "decode": ([1] * 5, [3, 40, 1, 300, 17], 12, 2),
    "decode_many": ([1] * 200, [20 + b % 90 for b in range(200)], 8, 1),
    "decode_cut": ([1], [20000], 6, 1),
    "drafts": ([8] * 3, [300, 2500, 8], 12, 3),
    "chunk_cut": ([100, 30], [9000, 31], 8, 2),
    "prompts": ([300, 127, 60], [300, 127, 60], 6, 2),
    "items": ([900, 800], [900, 800], 48, 8),
}


def _call(c, q):
    kc, vc, table, cu, lens = c.cuda()
    out = torch.zeros(q.shape, dtype=c.dt, device="cuda")
    lse = torch.zeros(c.N, c.Hq, dtype=torch.float32, device="cuda")
    gdn.gdn_paged_attn(q.cuda(), kc, vc, table, cu, lens, 0.1, max_q=max(c.new), max_kv=max(c.length), out=out, lse=lse)
    return out.float().cpu(), lse.cpu()


def _expect(c, out, lse, hit):
    """hit [N, Hq]: the rows that must be NaN; all others are finite."""
    assert bool(torch.isnan(out[hit]).all()) and bool(torch.isnan(lse[hit]).all())
    assert bool(torch.isfinite(out[~hit]).all()) and bool(torch.isfinite(lse[~hit]).all())
    assert gdn.gdn_check_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_nan_query(dtype, D, layout):
    new, length, Hq, Hk = LAYOUTS[layout]
    c = Paged(new, length, Hq, Hk, D, 64, dtype, seed=D)
    q = c.normal(c.N, Hq, D)
    hit = torch.zeros(c.N, Hq, dtype=torch.bool)
    for tok, head in ((0, 0), (c.N - 1, Hq - 1), (c.N // 2, Hq // 2)):
        q[tok, head] = NAN
        hit[tok, head] = True
    out, lse = _call(c, q)
    _expect(c, out, lse, hit)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_nan_key(dtype, D, layout, where):
    """One channel of one key of one head: the rows at or after its position, of the heads that read it."""
    new, length, Hq, Hk = LAYOUTS[layout]
    c = Paged(new, length, Hq, Hk, D, 64, dtype, seed=D + 1)
    q = c.normal(c.N, Hq, D)
    b, head, G = len(new) - 1, Hk - 1, Hq // Hk
    key = {"first": 0, "middle": length[b] // 2, "last": length[b] - 1}[where]
    c.kc[int(c.table[b, key // c.page]), head, key % c.page, 5] = NAN
    hit = torch.zeros(c.N, Hq, dtype=torch.bool)
    for tok, seq, pos in c.tokens():
        if seq == b and pos >= key:
            hit[tok, head * G:(head + 1) * G] = True
    out, lse = _call(c, q)
    _expect(c, out, lse, hit)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_nan_value(dtype, D, layout):
    """One channel of one cached value: that channel of the rows that see it (earlier rows of the sequence may
    have it too), and nothing else."""
    new, length, Hq, Hk = LAYOUTS[layout]
    c = Paged(new, length, Hq, Hk, D, 64, dtype, seed=D + 2)
    q = c.normal(c.N, Hq, D)
    b, head, G, key = len(new) - 1, Hk - 1, Hq // Hk, length[-1] // 2
    c.vc[int(c.table[b, key // c.page]), head, key % c.page, 7] = NAN
    out, lse = _call(c, q)
    may = torch.zeros(c.N, Hq, D, dtype=torch.bool)
    must = may.clone()
    for tok, seq, pos in c.tokens():
        if seq == b:
            may[tok, head * G:(head + 1) * G, 7] = True
            must[tok, head * G:(head + 1) * G, 7] = pos >= key
    assert bool(torch.isnan(out[must]).all()) and bool(torch.isfinite(out[~may]).all())
    assert bool(torch.isfinite(lse).all())
    assert gdn.gdn_check_device_error() == 0
