"""Refusals of the convolution, selective scan and plan calls, on the host: nothing reaches a GPU."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn
from gated_deltanet_gdn_gb300 import binding as b

OK, BAD, UNS = b.GDN_OK, b.GDN_ERR_INVALID_ARG, b.GDN_ERR_UNSUPPORTED
A = 1 << 20  # an aligned address that is never followed


@pytest.fixture(scope="module")
def lib():
    return gdn.load()


def _seqs(N=8, B=2, pool=2, cu=A, lens=None, slots=None):
    return b.GdnPacked(N, B, pool, cu, lens, slots)


def _row(p=A, rs=64, gs=0):
    return b.GdnRows(p, rs, gs)


BAD_SEQS = [(dict(N=-1), BAD), (dict(B=-1), BAD), (dict(pool=-1), BAD), (dict(N=(1 << 30) + 1), UNS), (dict(N=7, cu=None), BAD),
            (dict(B=0, cu=None), BAD), (dict(cu=A + 2), BAD), (dict(lens=A + 1), BAD), (dict(slots=A + 3), BAD)]


def _conv(lib, d, q, x=None, w=A, bias=None, s0=None, mq=4, y=None, sf=None):
    return lib.gdn_causal_conv_fwd(d, q, x or _row(), w, bias, s0, mq, y or _row(), sf, None)


def _conv_bwd(lib, d, q, x=None, w=A, bias=None, s0=None, dy=None, ds=None, dx=A, dw=A, db=None, ds0=None, ws=A):
    return lib.gdn_causal_conv_bwd(d, q, x or _row(), w, bias, s0, dy or _row(), ds, dx, dw, db, ds0, ws, None)


def test_conv_refusals(lib):
    def dims(C=64, taps=4, dtype=b.GDN_BF16, flags=0):
        return b.GdnConvDims(C, taps, dtype, flags)

    for kw, want in ((dict(C=0), BAD), (dict(taps=1), UNS), (dict(taps=5), UNS), (dict(dtype=4), UNS), (dict(flags=1), BAD),
                     (dict(flags=b.GDN_FLAG_DT_SOFTPLUS), BAD), (dict(C=1 << 25), UNS)):
        assert _conv(lib, dims(**kw), _seqs()) == want, kw
        assert _conv_bwd(lib, dims(**kw), _seqs()) == want, kw
        assert lib.gdn_causal_conv_workspace_bytes(dims(**kw), _seqs()) == 0
    for kw, want in BAD_SEQS:
        assert _conv(lib, dims(), _seqs(**kw)) == want, kw
        assert _conv_bwd(lib, dims(), _seqs(**kw)) == want, kw
    assert _conv(lib, None, _seqs()) == BAD and _conv(lib, dims(), None) == BAD
    for kw in (dict(w=None), dict(w=A + 1), dict(bias=A + 1), dict(s0=A + 1), dict(sf=A + 1), dict(mq=0), dict(x=_row(None)),
               dict(x=_row(A + 1)), dict(x=_row(A, -64)), dict(y=_row(None))):
        assert _conv(lib, dims(), _seqs(), **kw) == BAD, kw
    # a pool without slots has a row for every sequence
    assert _conv(lib, dims(), _seqs(pool=1), s0=A) == BAD and _conv(lib, dims(), _seqs(pool=1), sf=A) == BAD
    for kw in (dict(w=None), dict(dw=None), dict(dx=None), dict(db=A), dict(ws=None), dict(ws=A + 16), dict(dy=_row(None)), dict(ds=A + 1)):
        assert _conv_bwd(lib, dims(), _seqs(), **kw) == BAD, kw
    # the backward has no pools
    assert _conv_bwd(lib, dims(), _seqs(slots=A)) == BAD and _conv_bwd(lib, dims(), _seqs(lens=A)) == BAD
    none = _seqs(N=0, B=0, cu=None)
    assert _conv(lib, dims(), none, w=None) == OK and _conv_bwd(lib, dims(), none, w=None) == OK
    assert lib.gdn_causal_conv_workspace_bytes(dims(), _seqs()) >= 5 * 64 * 4


def test_scan_refusals(lib):
    def dims(D=64, G=2, S=16, dtype=b.GDN_BF16, flags=0):
        return b.GdnScanDims(D, G, S, dtype, flags)

    def parts(u=A, dt=A, z=None, B=A, C=A, a=A, skip=None, bias=None, h0=None, rs=64):
        return b.GdnScanParts(_row(u, rs), _row(dt, rs), _row(z, rs), _row(B, 32, 16), _row(C, 32, 16), a, skip, bias, h0)

    def fwd(d, q, p=None, mq=4, y=None, hf=None, res=None, ws=A):
        return lib.gdn_selective_scan_fwd(d, q, p or parts(), mq, y or _row(), hf, res, ws, None)

    def bwd(d, q, p=None, res=A, mq=4, dy=None, dh=None, g=None, ws=A):
        g = g or b.GdnScanGrads(A, A, None, A, A, A, None, None, None)
        return lib.gdn_selective_scan_bwd(d, q, p or parts(), res, mq, dy or _row(), dh, g, ws, None)

    for kw, want in ((dict(D=0), BAD), (dict(G=0), BAD), (dict(G=3), BAD), (dict(S=4), UNS), (dict(S=24), UNS), (dict(S=128), UNS),
                     (dict(dtype=3), UNS), (dict(flags=64), BAD), (dict(D=1 << 21), UNS)):
        assert fwd(dims(**kw), _seqs()) == want, kw
        assert bwd(dims(**kw), _seqs()) == want, kw
        assert lib.gdn_selective_scan_residual_bytes(dims(**kw), _seqs()) == 0
        assert lib.gdn_selective_scan_workspace_bytes(dims(**kw), _seqs(), 4) == 0
        assert lib.gdn_selective_scan_bwd_workspace_bytes(dims(**kw), _seqs(), 4) == 0
    for kw, want in BAD_SEQS:
        assert fwd(dims(), _seqs(**kw)) == want, kw
        assert bwd(dims(), _seqs(**kw)) == want, kw
    for kw in (dict(u=None), dict(dt=A + 1), dict(z=A + 1), dict(B=None), dict(C=A + 1), dict(a=None), dict(a=A + 4), dict(skip=A + 4),
               dict(bias=A + 8), dict(h0=A + 4), dict(rs=-1)):
        assert fwd(dims(), _seqs(), parts(**kw)) == BAD, kw
        assert bwd(dims(), _seqs(), parts(**kw)) == BAD, kw
    for kw in (dict(mq=0), dict(y=_row(None)), dict(y=_row(A + 1)), dict(hf=A + 4), dict(res=A + 4)):
        assert fwd(dims(), _seqs(), **kw) == BAD, kw
    assert fwd(dims(), _seqs(pool=1), parts(h0=A)) == BAD and fwd(dims(), _seqs(pool=1), hf=A) == BAD
    # residuals are the backward's, which has no pools
    assert fwd(dims(), _seqs(slots=A), res=A) == BAD and fwd(dims(), _seqs(lens=A), res=A) == BAD and bwd(dims(), _seqs(slots=A)) == BAD
    G = b.GdnScanGrads
    for kw in (dict(res=None), dict(mq=0), dict(dy=_row(None)), dict(dh=A + 4), dict(ws=None), dict(ws=A + 64),
               dict(g=G(None, A, None, A, A, A, None, None, None)), dict(g=G(A, None, None, A, A, A, None, None, None)),
               dict(g=G(A, A, A, A, A, A, None, None, None)), dict(g=G(A, A, None, None, A, A, None, None, None)),
               dict(g=G(A, A, None, A, A, None, None, None, None)), dict(g=G(A, A, None, A, A, A, A, None, None)),
               dict(g=G(A, A, None, A, A, A, None, A, None)), dict(g=G(A, A, None, A, A, A, None, None, A + 4)), dict(p=parts(z=A))):
        assert bwd(dims(), _seqs(), **kw) == BAD, kw
    none = _seqs(N=0, B=0, cu=None)
    assert fwd(dims(), none, parts(u=None)) == OK and bwd(dims(), none, parts(u=None)) == OK
    # a long sequence of few channels is split, one of many is not
    assert lib.gdn_selective_scan_workspace_bytes(dims(), _seqs(N=1 << 15, B=1), 1 << 15) > 0
    assert lib.gdn_selective_scan_workspace_bytes(dims(D=8192, G=1), _seqs(N=1 << 15, B=512), 64) == 0
    # states before every eight tokens, in whole quads of channels for every group
    assert lib.gdn_selective_scan_residual_bytes(dims(D=6, G=2), _seqs(N=16, B=2, cu=None)) == 2 * 1 * 8 * 16 * 4
    assert lib.gdn_selective_scan_residual_bytes(dims(D=6, G=2), _seqs(N=17, B=3)) == (17 // 8 + 3 + 1) * 8 * 16 * 4


def test_plan_refusals(lib):
    def dims(B=4, page=16, pages=8, free=10, top=32):
        return b.GdnPlanDims(B, page, pages, free, top)

    def out(cu=A, lens=A + 64, count=A + 128, requests=A + 192, positions=A + 256, slots=A + 512):
        return b.GdnPlanOut(cu, lens, count, requests, positions, slots)

    def plan(d, table=A + 1024, stride=8, lens=A + 2048, new=A + 2112, free=A + 2176, count=A + 2240, o=None):
        return lib.gdn_page_plan(d, table, stride, lens, new, free, count, o or out(), None)

    for kw, want in ((dict(B=-1), BAD), (dict(page=0), BAD), (dict(pages=-1), BAD), (dict(free=-1), BAD), (dict(top=-1), BAD),
                     (dict(B=8193), UNS), (dict(top=(1 << 30) + 1), UNS)):
        assert plan(dims(**kw)) == want, kw
    assert plan(None) == BAD
    for kw in (dict(table=None), dict(table=A + 2), dict(stride=7), dict(lens=None), dict(new=None), dict(free=None), dict(count=None),
               dict(count=A + 1), dict(o=out(cu=None)), dict(o=out(lens=None)), dict(o=out(count=None)), dict(o=out(requests=None)),
               dict(o=out(positions=None)), dict(o=out(slots=None)), dict(o=out(slots=A + 4)), dict(lens=A + 64), dict(new=A),
               dict(count=A + 128)):  # the last three: an output in an input's place
        assert plan(dims(), **kw) == BAD, kw


def test_bindings_refuse_cpu_tensors_and_wrong_shapes():
    x, w = torch.zeros(2, 4, 8), torch.zeros(8, 4)
    bc = torch.zeros(2, 4, 1, 16)
    ints = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: gdn.gdn_causal_conv_fwd(x, w), lambda: gdn.gdn_causal_conv_bwd(x, w, None, x), lambda: gdn.causal_conv(x, w),
                 lambda: gdn.gdn_selective_scan_fwd(x, x, torch.zeros(8, 16), bc, bc),
                 lambda: gdn.selective_scan(x, x, torch.zeros(8, 16), bc, bc),
                 lambda: gdn.gdn_page_plan(ints.view(3, 1), ints, ints, ints, ints[:1], page_size=16, max_tokens=4)):
        with pytest.raises(gdn.GdnError):
            call()
    for call in (lambda: gdn.gdn_causal_conv_fwd(None, w), lambda: gdn.gdn_causal_conv_fwd(x, 3),
                 lambda: gdn.gdn_page_plan(ints, ints, ints, ints, None, page_size=1, max_tokens=1)):
        with pytest.raises(TypeError):
            call()
