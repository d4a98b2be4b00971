"""GPU parity of gdn_block_norm_fwd / _bwd against the float64 formulas, the formulas
against central differences, and the kernels' gradient against differences of the forward."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn

from paged_reference import DT, UNIT

pytestmark = pytest.mark.gpu

EPS = 1e-6
FULL = dict(post=True, gate=True, residual=True, scale=True, pre=True)


def _act(g, sigmoid, ab=lambda t: t):
    """act(g) and its derivative (silu's is a sum whose terms cancel near g = -1.28)."""
    s = torch.sigmoid(g)
    return (s, s * (1 - s)) if sigmoid else (g * s, s + ab(g) * s * (1 - s))


def formulas(p, dh=None, dy=None, sigmoid=False, size=False):
    """The operator and its gradients in float64. size: each sum takes the magnitudes of its terms instead
    (the scale of the rounding errors of the same sums in fp32)."""
    ab = (lambda t: t.abs()) if size else (lambda t: t)
    minus = 1.0 if size else -1.0
    p = {k: (None if v is None else v.double()) for k, v in p.items()}
    x, gate, res, w1, sc, w2 = (p[k] for k in ("x", "gate", "residual", "w_post", "res_scale", "w_pre"))
    C = x.shape[-1]
    r1 = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / C + EPS)
    n = ab(x * r1 * w1) if w1 is not None else ab(x)
    a, d = _act(gate, sigmoid, ab) if gate is not None else (torch.ones(()).double(), torch.zeros(()).double())
    m = n * ab(a)
    s = ab(sc) if sc is not None else torch.ones(()).double()
    true_n = x * r1 * w1 if w1 is not None else x
    true_h = true_n * a * (sc if sc is not None else 1.0) + (res if res is not None else 0.0)
    h = m * s + (ab(res) if res is not None else 0.0)
    out = {"h": h}
    if w2 is not None:
        r2 = 1 / torch.sqrt((true_h * true_h).sum(-1, keepdim=True) / C + EPS)
        out["y"] = h * r2 * ab(w2)
    if dh is None and dy is None:
        return out
    D = ab(dh.double()) if dh is not None else torch.zeros_like(x)
    lead = tuple(range(x.dim() - 1))
    if w2 is not None:
        dy = dy.double()
        out["dw_pre"] = (ab(dy) * h * r2).sum(lead)
        t = ab(dy * w2)
        D = D + r2 * (t + minus * h * r2 ** 2 * (t * h).sum(-1, keepdim=True) / C)
    if res is not None:
        out["dresidual"] = D
    if sc is not None:
        out["dres_scale"] = (D * m).sum(lead)
    dm = D * s
    if gate is not None:
        out["dgate"] = dm * n * ab(d)
    dn = dm * ab(a)
    dx = dn
    if w1 is not None:
        out["dw_post"] = (dn * ab(x) * r1).sum(lead)
        u = dn * ab(w1)
        dx = r1 * (u + minus * ab(x) * r1 ** 2 * (u * ab(x)).sum(-1, keepdim=True) / C)
    out["dx"] = dx
    return out


def make(shape, dtype, parts, seed=0):
    g = torch.Generator().manual_seed(seed)
    C = shape[-1]

    def normal(*s, mean=0.0, std=1.0):
        return (torch.randn(*s, generator=g) * std + mean).to(DT[dtype])

    p = {"x": normal(*shape, mean=0.05, std=1.3), "gate": normal(*shape, std=1.5) if parts["gate"] else None,
         "residual": normal(*shape, std=2.0) if parts["residual"] else None,
         "w_post": normal(C, mean=1.0, std=0.2) if parts["post"] else None,
         "res_scale": normal(C, mean=0.5, std=0.2) if parts["scale"] else None,
         "w_pre": normal(C, mean=1.0, std=0.2) if parts["pre"] else None}
    return p, normal(*shape), normal(*shape) if parts["pre"] else None


def check(p, dh, dy, dtype, sigmoid=False, cuda=None):
    flags = gdn.GDN_FLAG_GATE_SIGMOID if sigmoid else 0
    d = cuda or {k: (None if v is None else v.cuda()) for k, v in p.items()}
    parts = {k: v for k, v in d.items() if k != "x"}
    h, y, stats = gdn.gdn_block_norm_fwd(d["x"], **parts, eps=EPS, flags=flags)
    grads = gdn.gdn_block_norm_bwd(d["x"], stats, None if dh is None else dh.cuda(), None if dy is None else dy.cuda(),
                                   **parts, eps=EPS, flags=flags)
    got = {"h": h, "y": y, **grads}
    ref, mag = formulas(p, dh, dy, sigmoid), formulas(p, dh, dy, sigmoid, size=True)
    for name, r in ref.items():
        # one rounding to the type, and fp32: a few dozen roundings along the chain plus a sum of up to C
        # (tree) or of a CTA's rows (serial, then over the CTAs), within 2^-16 of the terms' magnitudes
        tol = UNIT[dtype] * r.abs() + 2.0 ** -16 * mag[name] + 1e-30
        err = (got[name].double().cpu() - r).abs()
        assert bool((err <= tol).all()), (name, float((err / tol).max()))
    assert all(got[k] is None for k in ("y", "dgate", "dresidual", "dw_post", "dres_scale", "dw_pre") if k not in ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 64), (3, 2, 128), (700, 6, 128), (5, 1, 256), (33, 1, 1000), (7, 1, 1001),
                                   (2, 1, 1), (9, 3, 37), (400, 1, 2048), (3, 1, 4100), (311, 1, 6144), (2, 1, 8192),
                                   (2, 1, 8191), (1, 1, 4096)])
def test_all_parts_match_float64(dtype, shape):
    p, dh, dy = make(shape, dtype, FULL, seed=shape[-1])
    check(p, dh, dy, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [128, 520, 77])
@pytest.mark.parametrize("on", range(32))
def test_every_choice_of_parts(dtype, width, on):
    parts = {k: bool(on >> i & 1) for i, k in enumerate(("post", "gate", "residual", "scale", "pre"))}
    p, dh, dy = make((11, 2, width), dtype, parts, seed=on)
    check(p, dh, dy, dtype, sigmoid=bool(on & 1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("width", [1032, 2056, 2560, 3080, 5000, 6152, 8184])
def test_wide_rows_that_end_inside_a_step(dtype, gate, width):
    """Widths at which threads of the last step have no column, one row more than the SMs have CTAs."""
    parts = dict(FULL, gate=gate is not None)
    p, dh, dy = make((457, 1, width), dtype, parts, seed=width)
    check(p, dh, dy, dtype, sigmoid=gate == "sigmoid")


@pytest.mark.parametrize("width", [128, 640, 101])
def test_without_dh(width):
    p, _, dy = make((20, 1, width), "f32", FULL, seed=2)
    check(p, None, dy, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [128, 512])
def test_strided_rows(dtype, width):
    """x, gate and residual as slices of wider tensors, aligned to 16 bytes and not."""
    for off in (16, 3):
        p, dh, dy = make((13, 4, width), dtype, FULL, seed=off)
        cuda = {}
        for k, v in p.items():
            if v.dim() == 3:
                wide = torch.full((13, 5, width + 2 * off), 9.0, dtype=v.dtype, device="cuda")
                wide[:, 1:, off:off + width] = v.cuda()
                cuda[k] = wide[:, 1:, off:off + width]
            else:
                cuda[k] = v.cuda()
        check(p, dh, dy, dtype, cuda=cuda)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("parts", [("post", "gate"), ("post",), ("gate",)])
def test_many_strided_heads(dtype, parts):
    """Heads out of wider rows, more of them than are in work at once: every step of the walk over rows and
    groups, with groups left over."""
    R, G, C = 9001, 5, 64
    p, dh, dy = make((R, G, C), dtype, {k: k in parts for k in FULL}, seed=len(parts))
    cuda = {}
    for i, (k, v) in enumerate(p.items()):
        cuda[k] = None if v is None else v.cuda()
        if v is not None and v.dim() == 3:
            wide = torch.full((R, G + i + 1, C + 16), 9.0, dtype=v.dtype, device="cuda")
            wide[:, 1:G + 1, 8:8 + C] = v.cuda()
            cuda[k] = wide[:, 1:G + 1, 8:8 + C]
    check(p, dh, dy, dtype, cuda=cuda)


def test_formulas_against_central_differences():
    """float64: the gradients above are the derivatives of the forward above."""
    for sigmoid in (False, True):
        p, dh, dy = make((3, 2, 10), "f32", FULL, seed=5)
        p, dh, dy = {k: v.double() for k, v in p.items()}, dh.double(), dy.double()
        ref = formulas(p, dh, dy, sigmoid)

        def value(q):
            o = formulas(q, sigmoid=sigmoid)
            return float((o["h"] * dh).sum() + (o["y"] * dy).sum())

        names = dict(x="dx", gate="dgate", residual="dresidual", w_post="dw_post", res_scale="dres_scale", w_pre="dw_pre")
        g, e = torch.Generator().manual_seed(6), 1e-5
        for k, name in names.items():
            step = torch.randn(p[k].shape, generator=g, dtype=torch.float64)
            diff = (value({**p, k: p[k] + e * step}) - value({**p, k: p[k] - e * step})) / (2 * e)
            # truncation e^2 and cancellation 2^-52 / e, both under 1e-8 of values of order 100
            assert abs(diff - float((ref[name] * step).sum())) <= 1e-6 * (1 + abs(diff))


@pytest.mark.parametrize("width", [64, 300])
def test_kernel_gradients_against_differences_of_the_kernel(width):
    """Central differences of the fp32 forward along the gradient's own direction: step 2^-6 of unit length
    directions, rounding 2^-22 of the summed magnitudes over it, truncation of the order of the step squared."""
    p, dh, dy = make((6, 2, width), "f32", FULL, seed=7)
    d = {k: v.cuda() for k, v in p.items()}
    parts = {k: v for k, v in d.items() if k != "x"}
    _, _, stats = gdn.gdn_block_norm_fwd(d["x"], **parts, eps=EPS)
    grads = gdn.gdn_block_norm_bwd(d["x"], stats, dh.cuda(), dy.cuda(), **parts, eps=EPS)

    def value(q):
        x = q["x"]
        h, y, _ = gdn.gdn_block_norm_fwd(x, **{k: v for k, v in q.items() if k != "x"}, eps=EPS)
        return float((h.double() * dh.cuda().double()).sum() + (y.double() * dy.cuda().double()).sum())

    names = dict(x="dx", gate="dgate", residual="dresidual", w_post="dw_post", res_scale="dres_scale", w_pre="dw_pre")
    for k, name in names.items():
        gr = grads[name].double()
        step = gr / gr.norm()
        e = 2.0 ** -4
        diff = (value({**d, k: (d[k].double() + e * step).float()}) - value({**d, k: (d[k].double() - e * step).float()})) / (2 * e)
        assert abs(diff - float(gr.norm())) <= 1e-2 * float(gr.norm()), (name, diff, float(gr.norm()))


def test_autograd_and_repeat_bitwise():
    p, dh, dy = make((64, 2, 128), "bf16", FULL, seed=8)
    d = {k: v.cuda().requires_grad_() for k, v in p.items()}
    h, y = gdn.block_norm(d["x"], **{k: v for k, v in d.items() if k != "x"}, eps=EPS)
    a = torch.autograd.grad([h, y], list(d.values()), [dh.cuda(), dy.cuda()], retain_graph=True)
    b = torch.autograd.grad([h, y], list(d.values()), [dh.cuda(), dy.cuda()])
    raw = {k: v.detach() for k, v in d.items()}
    parts = {k: v for k, v in raw.items() if k != "x"}
    _, _, stats = gdn.gdn_block_norm_fwd(raw["x"], **parts, eps=EPS)
    g = gdn.gdn_block_norm_bwd(raw["x"], stats, dh.cuda(), dy.cuda(), **parts, eps=EPS)
    for u, v, w in zip(a, b, (g[n] for n in ("dx", "dgate", "dresidual", "dw_post", "dres_scale", "dw_pre"))):
        assert torch.equal(u, v) and torch.equal(u, w)


def test_no_rows():
    x = torch.empty(0, 3, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    h, y, stats = gdn.gdn_block_norm_fwd(x, w_pre=w)
    assert h.shape == y.shape == x.shape
    g = gdn.gdn_block_norm_bwd(x, stats, x, x, w_pre=w)
    assert bool((g["dw_pre"] == 0).all())


def test_leading_dimensions_fold():
    p, dh, dy = make((6, 4, 64), "f32", FULL, seed=10)
    d = {k: v.cuda() for k, v in p.items()}
    parts = {k: v for k, v in d.items() if k != "x"}
    h, y, _ = gdn.gdn_block_norm_fwd(d["x"], **parts)
    four = {k: (v.view(2, 3, 4, 64) if v.dim() == 3 else v) for k, v in d.items()}
    h4, y4, _ = gdn.gdn_block_norm_fwd(four["x"], **{k: v for k, v in four.items() if k != "x"})
    assert h4.shape == (2, 3, 4, 64) and torch.equal(h4.view_as(h), h) and torch.equal(y4.view_as(y), y)
