"""GPU parity of gdn_kv_append against the float64 rotation: rows, pages, strides, tokens
that are not kept, errors; and that nothing else in the cache changes."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn

from paged_reference import DT, UNIT, Paged, rotated

pytestmark = pytest.mark.gpu


def _tables(positions, rot):
    ang = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rot // 2) * 2.0 / rot)
    return ang.cos().float(), ang.sin().float()


def _close(x, ref, mag, dtype):
    """One rounding to the type, and the fp32 products and sum (three roundings of 2^-24)."""
    return bool(((x.double().cpu() - ref).abs() <= UNIT[dtype] * ref.abs() + 3 * 2.0 ** -24 * mag).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,rot,pairs", [(128, 128, False), (128, 64, True), (64, 16, False), (64, 64, True),
                                         (128, 0, False)])
@pytest.mark.parametrize("new,length,Hq,Hk,page", [([1, 1, 1], [1, 16, 333], 6, 2, 16), ([5, 0, 40], [5, 9, 100], 1, 1, 48),
                                                   ([300], [700], 40, 8, 64)])
@pytest.mark.parametrize("rows_first", [False, True])
def test_matches_float64(dtype, D, rot, pairs, new, length, Hq, Hk, page, rows_first):
    c = Paged(new, length, Hq, Hk, D, page, dtype, seed=rot + D, rows_first=rows_first)
    qkv = c.normal(c.N, Hq + 2 * Hk, D)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    kc, vc, table, cu, lens = c.cuda()
    dev = qkv.cuda()
    cos, sin = _tables(max(length), rot) if rot else (torch.ones(1, 0), torch.zeros(1, 0))
    tab = dict(cos=cos.cuda(), sin=sin.cuda()) if rot else {}
    qo = gdn.gdn_kv_append(dev[:, Hq:Hq + Hk], dev[:, Hq + Hk:], kc, vc, table, cu, lens, q=dev[:, :Hq],
                           flags=gdn.GDN_FLAG_ROPE_PAIRS if pairs else 0, **tab)
    pos = [p for _, _, p in c.tokens()]
    if rot:
        qr, qm = rotated(q, pos, cos, sin, pairs)
        kr, km = rotated(k, pos, cos, sin, pairs)
    else:
        qr, qm, kr, km = q.double(), q.double().abs(), k.double(), k.double().abs()
    assert _close(qo, qr, qm, dtype)
    kc, vc = kc.cpu(), vc.cpu()
    kx, vx = c.kc.clone(), c.vc.clone()
    for (tok, b, p) in c.tokens():
        pg, row = int(c.table[b, p // page]), p % page
        assert _close(kc[pg, :, row], kr[tok], km[tok], dtype)
        assert torch.equal(vc[pg, :, row], v[tok])
        kx[pg, :, row], vx[pg, :, row] = kc[pg, :, row], vc[pg, :, row]
    # every other row is what it was (NaN included)
    assert torch.equal(torch.nan_to_num(kc.float(), nan=1e9), torch.nan_to_num(kx.float(), nan=1e9))
    assert torch.equal(torch.nan_to_num(vc.float(), nan=1e9), torch.nan_to_num(vx.float(), nan=1e9))
    assert gdn.gdn_check_device_error() == 0


def test_q_in_place_and_without_q():
    c = Paged([4], [50], 4, 2, 64, 16, "bf16", seed=1)
    cos, sin = (t.cuda() for t in _tables(50, 64))
    q, k, v = c.normal(4, 4, 64).cuda(), c.normal(4, 2, 64).cuda(), c.normal(4, 2, 64).cuda()
    kc, vc, table, cu, lens = c.cuda()
    assert gdn.gdn_kv_append(k, v, kc, vc, table, cu, lens, cos=cos, sin=sin) is None
    first = kc.clone()
    out = gdn.gdn_kv_append(k, v, kc, vc, table, cu, lens, q=q, cos=cos, sin=sin)
    same = gdn.gdn_kv_append(k, v, kc, vc, table, cu, lens, q=q, q_out=q, cos=cos, sin=sin)
    assert same is q and torch.equal(q, out)
    assert torch.equal(torch.nan_to_num(kc.float(), nan=9.), torch.nan_to_num(first.float(), nan=9.))


def test_tokens_before_position_zero_and_padding_are_not_kept():
    c = Paged([3, 2], [1, 20], 2, 2, 64, 16, "f32", seed=2)
    cos, sin = (t.cuda() for t in _tables(20, 32))
    N = 8  # three rows of padding
    q, k, v = (c.normal(N, 2, 64) for _ in range(3))
    kc, vc, table, cu, lens = c.cuda()
    q_out = torch.full((N, 2, 64), 5.0, device="cuda")
    gdn.gdn_kv_append(k.cuda(), v.cuda(), kc, vc, table, cu, lens, q=q.cuda(), q_out=q_out, cos=cos, sin=sin)
    q_out = q_out.cpu()
    assert torch.equal(q_out[:2], q[:2])  # positions -2, -1: not turned, not kept
    assert bool((q_out[5:] == 5).all())
    kept = (vc.cpu()[:, 0, :, 0] != c.vc[:, 0, :, 0]) & ~torch.isnan(vc.cpu()[:, 0, :, 0])
    assert int(kept.sum()) == 3
    assert gdn.gdn_check_device_error() == 0


def test_bad_pages_lengths_and_positions_are_reported_and_not_stored():
    c = Paged([1], [40], 2, 1, 64, 16, "bf16", seed=3)
    k, v = c.normal(1, 1, 64).cuda(), c.normal(1, 1, 64).cuda()
    kc, vc, table, cu, lens = c.cuda()
    before = torch.nan_to_num(vc.float(), nan=9.0)
    cos, sin = (t.cuda() for t in _tables(30, 64))
    bad = table.clone()
    bad[0, 2] = c.count
    for tab, ln, rope in ((bad, lens, {}), (table, lens + 1000, {}), (table, lens, dict(cos=cos, sin=sin))):
        gdn.gdn_kv_append(k, v, kc, vc, tab, cu, ln, **rope)
        assert gdn.gdn_check_device_error() == gdn.binding.GDN_ERR_INTERNAL
        assert torch.equal(torch.nan_to_num(vc.float(), nan=9.0), before)


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements: the last page is the one that is written and read."""
    page, D, Hk = 256, 128, 8
    count = (1 << 31) // (page * D * Hk) + 3
    kc = torch.empty(count, Hk, page, D, dtype=DT["bf16"], device="cuda")
    vc = torch.empty_like(kc)
    table = torch.tensor([[count - 1]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    lens = torch.tensor([5], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(5, Hk, D, generator=g).to(DT["bf16"]).cuda() for _ in range(2))
    gdn.gdn_kv_append(k, v, kc, vc, table, cu, lens)
    assert torch.equal(kc[count - 1, :, :5].transpose(0, 1), k) and torch.equal(vc[count - 1, :, :5].transpose(0, 1), v)
    q = torch.randn(5, 32, D, generator=g).to(DT["bf16"]).cuda()
    for max_q in (1, 5):
        out = gdn.gdn_paged_attn(q, kc, vc, table, cu, lens, max_q=max_q, max_kv=5).double()
        s = torch.einsum("nhgd,khd->nhgk", q.double().view(5, Hk, 4, D), k.double()) * D ** -0.5
        s = s.masked_fill(torch.arange(5, device="cuda")[None, :] > torch.arange(5, device="cuda")[:, None, None, None], -float("inf"))
        ref = torch.einsum("nhgk,khd->nhgd", torch.softmax(s, -1), v.double()).reshape(5, 32, D)
        assert float((out - ref).abs().max()) <= 2 * UNIT["bf16"] * float(v.double().abs().max()) * 1.1
    assert gdn.gdn_check_device_error() == 0
