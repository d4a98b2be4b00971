"""Packed rows whose offsets do not begin at zero: the convolution and the scan over part of a batch, against 64 bits. Rows of
no sequence hold NaN, become zeros in new outputs, stay as they were in given ones, and have zero gradients."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn
from tests.mixer_reference import conv_seq, over_channels, scan_seq, within

pytestmark = pytest.mark.gpu
SILU, SOFT = gdn.GDN_FLAG_CONV_SILU, gdn.GDN_FLAG_DT_SOFTPLUS

# offsets, rows
OFFSETS = [([40, 80, 100], 100), ([40, 80, 100], 117), ([5, 9, 30, 30, 31], 31), ([16, 17], 40), ([33, 33], 50), ([7], 20), ([50], 50),
           ([300, 302, 303, 305], 310)]


def _normal(gen, *shape, dtype=torch.float32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)


def _rest(at, rows, *tensors):
    """Mask of the rows of no sequence, where the tensors become NaN."""
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[at[0]:at[-1]] = False
    for t in tensors:
        t[rest] = float("nan")
    return rest


@pytest.mark.parametrize("bound", [None, 4])  # runs of a sequence's tokens, and whole sequences
@pytest.mark.parametrize("C,dtype", [(64, torch.bfloat16), (37, torch.float32)])
@pytest.mark.parametrize("at,rows", OFFSETS)
def test_convolution(at, rows, C, dtype, bound):
    gen = torch.Generator(device="cuda").manual_seed(sum(at) + C)
    n, cu = len(at) - 1, torch.tensor(at, dtype=torch.int32, device="cuda")
    x, w, bias, s0 = (_normal(gen, *s, dtype=dtype) for s in ((rows, C), (C, 4), (C,), (n, 3, C)))
    rest = _rest(at, rows, x)
    y, state = gdn.gdn_causal_conv_fwd(x, w, bias, state0=s0, cu_seqlens=cu, max_q=bound, flags=SILU)
    given = torch.full((rows, C), 7.0, dtype=dtype, device="cuda")
    gdn.gdn_causal_conv_fwd(x, w, bias, state0=s0, cu_seqlens=cu, max_q=bound, out=given, flags=SILU)
    assert not bool(y[rest].any()) and bool((given[rest] == 7).all()) and torch.equal(given[~rest], y[~rest])
    for b in range(n):
        r = slice(at[b], at[b + 1])
        ref = conv_seq(x[r], w, bias, s0[b], True)
        within("y", y[r], *ref["y"])
        assert torch.equal(state[b].double(), ref["state"][0])


@pytest.mark.parametrize("C,dtype", [(64, torch.bfloat16), (37, torch.float32)])
@pytest.mark.parametrize("at,rows", OFFSETS)
def test_convolution_gradients(at, rows, C, dtype):
    gen = torch.Generator(device="cuda").manual_seed(sum(at) + C + 1)
    n, cu = len(at) - 1, torch.tensor(at, dtype=torch.int32, device="cuda")
    x, dy, w, bias, s0, ds = (_normal(gen, *s, dtype=dtype) for s in ((rows, C), (rows, C), (C, 4), (C,), (n, 3, C), (n, 3, C)))
    rest = _rest(at, rows, x, dy)
    leaves = [t.requires_grad_() for t in (x, w, bias, s0)]
    y, state = gdn.causal_conv(*leaves, cu_seqlens=cu, flags=SILU)
    dx, dw, db, dst = torch.autograd.grad([y, state], leaves, [dy, ds])
    assert not bool(dx[rest].any())
    vw, ew, vb, eb = (torch.zeros(*s, dtype=torch.float64, device="cuda") for s in ((C, 4), (C, 4), (C,), (C,)))
    for b in range(n):
        r = slice(at[b], at[b + 1])
        ref = conv_seq(x[r], w, bias, s0[b], True, dy[r], ds[b])
        within("dx", dx[r], *ref["dx"])
        within("dstate0", dst[b], *ref["dstate0"])
        vw, ew, vb, eb = vw + ref["dweight"][0], ew + ref["dweight"][1], vb + ref["dbias"][0], eb + ref["dbias"][1]
    within("dweight", dw, vw, ew * 1.01)  # and the order of a few sequences' sums
    within("dbias", db, vb, eb * 1.01)


def _scan_inputs(gen, rows, D, G, S, dtype):
    return dict(u=_normal(gen, rows, D, dtype=dtype), dt=_normal(gen, rows, D, dtype=dtype, std=0.7),
                A=-torch.arange(1, S + 1, device="cuda") * torch.exp(_normal(gen, D, S, std=0.2)), B=_normal(gen, rows, G, S, dtype=dtype),
                C=_normal(gen, rows, G, S, dtype=dtype), D=_normal(gen, D), z=_normal(gen, rows, D, dtype=dtype),
                dt_bias=_normal(gen, D, mean=-3.0))


def _cut(s, r, **more):
    return dict({k: s[k][r] for k in ("u", "dt", "B", "C", "z")}, A=s["A"], D=s["D"], bias=s["dt_bias"], **more)


# channels, groups, states; with 3000 rows the sequences are cut into chunks
SCANS = [(at, rows, D, G, S, dtype) for at, rows in OFFSETS for D, G, S, dtype in ((40, 1, 16, torch.bfloat16), (14, 2, 64, torch.float32))]
SCANS += [([1000, 2900, 2901], 3000, 32, 1, 16, torch.float32), ([77, 1500, 1500, 3000], 3000, 20, 1, 8, torch.bfloat16)]


@pytest.mark.parametrize("bound", [None, 2])  # tiles of tokens, and token by token
@pytest.mark.parametrize("at,rows,D,G,S,dtype", SCANS)
def test_scan(at, rows, D, G, S, dtype, bound):
    gen = torch.Generator(device="cuda").manual_seed(sum(at) + D)
    n, cu = len(at) - 1, torch.tensor(at, dtype=torch.int32, device="cuda")
    s, h0 = _scan_inputs(gen, rows, D, G, S, dtype), _normal(gen, n, D, S)
    rest = _rest(at, rows, s["u"], s["dt"], s["B"], s["C"], s["z"])
    if rows == 3000 and bound is None:
        dims, seqs = gdn.binding.GdnScanDims(D, G, S, gdn.GDN_F32, SOFT), gdn.binding.GdnPacked(rows, n, n, 1 << 20, None, None)
        assert gdn.load().gdn_selective_scan_workspace_bytes(dims, seqs, rows) > 0
    y, h, _ = gdn.gdn_selective_scan_fwd(**s, h0=h0, cu_seqlens=cu, max_q=bound, flags=SOFT)
    given = torch.full((rows, D), 7.0, dtype=dtype, device="cuda")
    gdn.gdn_selective_scan_fwd(**s, h0=h0, cu_seqlens=cu, max_q=bound, out=given, flags=SOFT)
    assert not bool(y[rest].any()) and bool((given[rest] == 7).all()) and torch.equal(given[~rest], y[~rest])
    for b in range(n):
        r = slice(at[b], at[b + 1])
        ref = scan_seq(**_cut(s, r, h0=h0[b]))
        within("y", y[r], *ref["y"])
        within("h", h[b], *ref["h"])


@pytest.mark.parametrize("at,rows,D,G,S,dtype", SCANS)
def test_scan_gradients(at, rows, D, G, S, dtype):
    gen = torch.Generator(device="cuda").manual_seed(sum(at) + D + 1)
    n, cu = len(at) - 1, torch.tensor(at, dtype=torch.int32, device="cuda")
    s, h0, dh = _scan_inputs(gen, rows, D, G, S, dtype), _normal(gen, n, D, S), _normal(gen, n, D, S)
    dy = _normal(gen, rows, D, dtype=dtype)
    rest = _rest(at, rows, s["u"], s["dt"], s["B"], s["C"], s["z"], dy)
    _, _, kept = gdn.gdn_selective_scan_fwd(**s, h0=h0, cu_seqlens=cu, flags=SOFT, save=True)
    g = gdn.gdn_selective_scan_bwd(s["u"], s["dt"], s["A"], s["B"], s["C"], dy, kept, D=s["D"], z=s["z"], dt_bias=s["dt_bias"], dh_final=dh,
                                   need_dh0=True, cu_seqlens=cu, flags=SOFT)
    for k in ("du", "ddt", "dz", "dB", "dC"):
        assert not bool(g[k][rest].any()), k
    sums = {k: (torch.zeros(*v, dtype=torch.float64, device="cuda"),) * 2 for k, v in (("dA", (D, S)), ("dD", (D,)), ("ddt_bias", (D,)))}
    for b in range(n):
        r = slice(at[b], at[b + 1])
        if at[b] == at[b + 1]:
            assert torch.equal(g["dh0"][b], dh[b])
            continue
        ref = scan_seq(**_cut(s, r, h0=h0[b], dy=dy[r], dh=dh[b]))
        for k in ("du", "ddt", "dz"):
            within(k, g[k][r], *ref[k])
        within("dB", g["dB"][r], *over_channels(ref["dB"], G))
        within("dC", g["dC"][r], *over_channels(ref["dC"], G))
        within("dh0", g["dh0"][b], *ref["dh0"])
        for k in sums:
            sums[k] = (sums[k][0] + ref[k][0], sums[k][1] + ref[k][1] * 1.01)  # and the order of a few sequences' sums
    for k in sums:
        within(k, g[k], *sums[k])
