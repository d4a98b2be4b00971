"""Refusals of the paged cache and block norm calls, on the host: nothing reaches a GPU."""
import ctypes

import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn
from gated_deltanet_gdn_gb300 import binding as b

OK, BAD, UNS = b.GDN_OK, b.GDN_ERR_INVALID_ARG, b.GDN_ERR_UNSUPPORTED
A = 1 << 20  # an aligned address that is never followed


def _dims(**kw):
    d = dict(N=4, B=2, Hq=8, Hk=2, D=128, page_size=64, num_pages=10, max_pages=4, dtype=b.GDN_BF16, flags=0)
    d.update(kw)
    return b.GdnPagedDims(*d.values())


def _cache(**kw):
    d = dict(k=A, v=A, k_page_stride=16384, k_head_stride=8192, k_row_stride=128, v_page_stride=16384,
             v_head_stride=8192, v_row_stride=128, page_table=A, page_table_stride=4, cu_seqlens=A, kv_lens=A)
    d.update(kw)
    return b.GdnPagedCache(*d.values())


def _tok(p=A, ts=1024, hs=128):
    return b.GdnTokens(p, ts, hs)


BAD_DIMS = [(dict(N=-1), BAD), (dict(B=-1), BAD), (dict(Hk=0), BAD), (dict(Hq=7), BAD), (dict(D=96), UNS),
            (dict(page_size=24), UNS), (dict(page_size=0), BAD), (dict(dtype=5), UNS), (dict(flags=1), BAD),
            (dict(N=1 << 30), UNS), (dict(num_pages=0), BAD), (dict(max_pages=0), BAD)]
BAD_CACHE = [dict(k=None), dict(v=A + 8), dict(page_table=None), dict(cu_seqlens=A + 2), dict(kv_lens=None),
             dict(k_row_stride=100), dict(v_head_stride=-128), dict(k_page_stride=3), dict(page_table_stride=-1)]


@pytest.fixture(scope="module")
def lib():
    return gdn.load()


def _append(lib, d, c, k=None, v=None, q=None, qo=None, cos=A, sin=A, positions=100, rot=64):
    return lib.gdn_kv_append(d, c, k or _tok(), v or _tok(), q, qo, cos, sin, positions, rot, None)


def _attn(lib, d, c, q=None, scale=0.1, mq=2, mk=100, out=None, lse=None, ws=A):
    return lib.gdn_paged_attn(d, c, q or _tok(), scale, mq, mk, out or _tok(), lse, ws, None)


def test_paged_refusals(lib):
    for kw, want in BAD_DIMS:
        assert _append(lib, _dims(**kw), _cache()) == want, kw
        assert _attn(lib, _dims(**kw), _cache()) == want, kw
    assert _attn(lib, None, _cache()) == BAD and _append(lib, None, _cache()) == BAD
    for kw in BAD_CACHE:
        assert _append(lib, _dims(), _cache(**kw)) == BAD, kw
        assert _attn(lib, _dims(), _cache(**kw)) == BAD, kw
    assert _attn(lib, _dims(), None) == BAD
    for t in (_tok(None), _tok(A + 4), _tok(A, 1000 + 4), _tok(A, 1024, -128)):
        assert _append(lib, _dims(), _cache(), k=t) == BAD
        assert _append(lib, _dims(), _cache(), v=t) == BAD
        assert _attn(lib, _dims(), _cache(), q=t) == BAD
        assert _attn(lib, _dims(), _cache(), out=t) == BAD
    assert _append(lib, _dims(), _cache(), q=_tok(), qo=None) == BAD
    assert _append(lib, _dims(), _cache(), q=_tok(A + 4), qo=_tok()) == BAD
    for kw in (dict(rot=8), dict(rot=-16), dict(rot=144), dict(cos=None), dict(sin=A + 4), dict(positions=0)):
        assert _append(lib, _dims(), _cache(), **kw) == BAD, kw
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(mq=0), dict(mk=0), dict(ws=None),
               dict(ws=A + 16), dict(lse=A + 1)):
        assert _attn(lib, _dims(), _cache(), **kw) == BAD, kw
    # nothing to do: nothing is looked at
    for kw in (dict(N=0), dict(B=0)):
        assert _attn(lib, _dims(**kw), None) == OK and _append(lib, _dims(**kw), None) == OK


def test_workspace_sizes(lib):
    f = lib.gdn_paged_attn_workspace_bytes
    assert f(_dims(), 1, 100) > 0
    for d, mq, mk in ((None, 1, 1), (_dims(D=96), 1, 1), (_dims(N=0), 1, 1), (_dims(), 0, 1), (_dims(), 1, 0)):
        assert f(d, mq, mk) == 0
    g = lib.gdn_block_norm_workspace_bytes
    assert g(b.GdnNormDims(5, 1, 100, 0, 0, 1e-6)) > 0
    assert g(b.GdnNormDims(0, 1, 100, 0, 0, 1e-6)) == 0 and g(None) == 0


def _norm(R=4, G=2, C=128, dtype=b.GDN_F32, flags=0, eps=1e-6):
    return b.GdnNormDims(R, G, C, dtype, flags, eps)


def _parts(x=A, gate=None, residual=None, w_post=None, res_scale=None, w_pre=None):
    return b.GdnNormParts(b.GdnRows(x, 256, 128), b.GdnRows(gate, 256, 128), b.GdnRows(residual, 256, 128), w_post,
                          res_scale, w_pre)


def test_norm_refusals(lib):
    fwd, bwd = lib.gdn_block_norm_fwd, lib.gdn_block_norm_bwd
    row = b.GdnRows(A, 256, 128)
    grads = b.GdnNormGrads(A, None, None, None, None, None)
    for kw, want in ((dict(R=-1), BAD), (dict(G=0), BAD), (dict(C=0), BAD), (dict(C=8193), UNS), (dict(dtype=3), UNS),
                     (dict(flags=4), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
                     (dict(R=1 << 30, G=4), UNS)):
        assert fwd(_norm(**kw), _parts(), A, None, A, None) == want, kw
        assert bwd(_norm(**kw), _parts(), A, row, None, grads, A, None) == want, kw
    assert fwd(None, _parts(), A, None, A, None) == BAD
    for p, h, y, st in ((None, A, None, A), (_parts(x=None), A, None, A), (_parts(x=A + 2), A, None, A),
                        (_parts(), None, None, A), (_parts(), A, None, None), (_parts(), A, A, A),
                        (_parts(w_pre=A), A, None, A), (_parts(w_post=A + 1), A, None, A), (_parts(), A + 1, None, A),
                        (_parts(gate=A + 2), A, None, A)):
        assert fwd(_norm(), p, h, y, st, None) == BAD
    assert fwd(_norm(R=0), None, None, None, None, None) == OK
    ok = dict(p=_parts(), st=A, dh=row, dy=None, g=grads, ws=A)
    for kw in (dict(p=None), dict(st=None), dict(dh=None), dict(dy=row), dict(g=None), dict(ws=None), dict(ws=A + 64),
               dict(p=_parts(w_pre=A)), dict(g=b.GdnNormGrads(None)), dict(g=b.GdnNormGrads(A, A)),
               dict(g=b.GdnNormGrads(A, None, A)), dict(g=b.GdnNormGrads(A, None, None, A)),
               dict(g=b.GdnNormGrads(A, None, None, None, A)), dict(g=b.GdnNormGrads(A, None, None, None, None, A)),
               dict(g=b.GdnNormGrads(A + 2)), dict(dh=b.GdnRows(A, -4, 0))):
        a = {**ok, **kw}
        assert bwd(_norm(), a["p"], a["st"], a["dh"], a["dy"], a["g"], a["ws"], None) == BAD, kw
    assert bwd(_norm(R=0), None, None, None, None, grads, None, None) == OK


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    t = torch.zeros(4, 2, 64)
    cache = torch.zeros(3, 2, 16, 64)
    ints = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_paged_attn(t, cache, cache, *ints)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_kv_append(t, t, cache, cache, *ints)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_block_norm_fwd(t)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_block_norm_fwd(torch.zeros(8))


def test_profile_names_cover_the_kernels(lib):
    names = [gdn.gdn_kernel_name(i) for i in range(b.KERNEL_COUNT)]
    assert len(set(names)) == b.KERNEL_COUNT and all(names) and gdn.gdn_kernel_name(b.KERNEL_COUNT) == ""
    assert ctypes.sizeof(b.GdnPagedDims) == 40
