"""Causal convolution against 64 bits: packed and batched, states in pools, odd sizes, gradients, refusals."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn
from tests.mixer_reference import conv_seq, within

pytestmark = pytest.mark.gpu
SILU = gdn.GDN_FLAG_CONV_SILU


def _normal(gen, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _packed(lens, pad=0):
    cu = torch.tensor([sum(lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    return cu, sum(lens) + pad


# lengths, rows behind, channels, taps, silu, bias, states
PACKED = [([1] * 5, 0, 768, 4, True, False, True), ([1, 2, 3, 4, 5], 3, 64, 4, True, True, True), ([0, 7, 0, 1, 0], 9, 40, 3, True, True, True),
          ([33, 129, 1], 70, 37, 2, False, True, True), ([300, 17], 1, 1001, 4, True, False, False), ([1], 0, 1, 4, True, True, True),
          ([64, 64, 65], 0, 96, 3, False, False, True), ([], 20, 16, 4, True, False, False), ([8, 16, 24], 40, 128, 4, True, True, True)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,pad,C,taps,silu,with_bias,with_state", PACKED)
def test_packed_forward(lens, pad, C, taps, silu, with_bias, with_state, dtype):
    gen = torch.Generator(device="cuda").manual_seed(sum(lens) * 7 + C)
    cu, rows = _packed(lens, pad)
    n, pool = len(lens), len(lens) + 4
    x = _normal(gen, rows, C, dtype=dtype)
    w, bias = _normal(gen, C, taps, dtype=dtype), _normal(gen, C, dtype=dtype) if with_bias else None
    states = _normal(gen, pool, taps - 1, C, dtype=dtype) if with_state else None
    slots = torch.randperm(pool, generator=gen, device="cuda")[:n].to(torch.int32)
    if n > 2:
        slots[1] = -1  # a sequence without a state
    past = [0 if b == n - 1 and n > 1 else 5 for b in range(n)]
    kv = torch.tensor([p + v for p, v in zip(past, lens)], dtype=torch.int32, device="cuda")
    before = torch.full((pool, taps - 1, C), 3.0, dtype=dtype, device="cuda")
    after = before.clone()
    y, got = gdn.gdn_causal_conv_fwd(x, w, bias, state0=states, state_final=after, slots=slots, cu_seqlens=cu, kv_lens=kv,
                                     max_q=max(lens + [1]), flags=SILU if silu else 0)
    assert got is after
    written = set()
    for b in range(n):
        slot, r = int(slots[b]), slice(int(cu[b]), int(cu[b + 1]))
        zero = torch.zeros(taps - 1, C, dtype=dtype, device="cuda")
        s0 = states[slot] if with_state and slot >= 0 and past[b] > 0 else zero
        ref = conv_seq(x[r], w, bias, s0, silu)
        within("y", y[r], *ref["y"])
        if slot >= 0:
            assert torch.equal(after[slot].double(), ref["state"][0])
            written.add(slot)
    for slot in set(range(pool)) - written:
        assert torch.equal(after[slot], before[slot])
    assert not bool(y[sum(lens):].any())
    # in place, and into given rows with gaps between them: the rows behind the last sequence are left alone
    wide = torch.full((rows, C + 8), 7.0, dtype=dtype, device="cuda")
    if with_state:
        own = states.clone()
        y2, s2 = gdn.gdn_causal_conv_fwd(x, w, bias, state0=own, state_final=own, slots=slots, cu_seqlens=cu, kv_lens=kv,
                                         out=wide[:, :C], flags=SILU if silu else 0)
        assert torch.equal(y2[:sum(lens)], y[:sum(lens)]) and bool((wide[sum(lens):] == 7).all()) and bool((wide[:, C:] == 7).all())
        for slot in range(pool):
            assert torch.equal(own[slot], after[slot] if slot in written else states[slot])
    assert gdn.gdn_check_device_error() == 0


# sequences, tokens, channels, taps, silu, bias, state, gradient of the state
TRAIN = [(2, 40, 768, 4, True, False, False, False), (3, 17, 37, 3, True, True, True, True), (1, 1, 64, 4, True, True, True, True),
         (2, 2, 12, 4, False, True, True, True), (1, 700, 24, 2, True, False, True, False), (4, 129, 101, 4, False, True, False, True),
         (5, 3, 8, 4, True, True, True, True), (1, 9001, 20, 3, True, True, True, True), (3, 1000, 136, 4, False, True, False, False)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,T,C,taps,silu,with_bias,with_state,with_dstate", TRAIN)
def test_training(n, T, C, taps, silu, with_bias, with_state, with_dstate, dtype):
    gen = torch.Generator(device="cuda").manual_seed(n * T + C)
    x, dy = _normal(gen, n, T, C, dtype=dtype), _normal(gen, n, T, C, dtype=dtype)
    w, bias = _normal(gen, C, taps, dtype=dtype), _normal(gen, C, dtype=dtype) if with_bias else None
    s0 = _normal(gen, n, taps - 1, C, dtype=dtype) if with_state else None
    ds = _normal(gen, n, taps - 1, C, dtype=dtype) if with_dstate else None
    leaves = [t.requires_grad_() for t in (x, w, bias, s0) if t is not None]
    y, state = gdn.causal_conv(x, w, bias, s0, flags=SILU if silu else 0)
    outs, gs = ([y, state], [dy, ds]) if with_dstate else ([y], [dy])
    grads = dict(zip([n_ for n_, t in (("dx", x), ("dweight", w), ("dbias", bias), ("dstate0", s0)) if t is not None],
                     torch.autograd.grad(outs, leaves, gs)))
    sums = {}
    for b in range(n):
        zero = torch.zeros(taps - 1, C, dtype=dtype, device="cuda")
        ref = conv_seq(x[b], w, bias, zero if s0 is None else s0[b], silu, dy[b], None if ds is None else ds[b])
        within("y", y[b].detach(), *ref["y"])
        assert torch.equal(state[b].detach().double(), ref["state"][0])
        within("dx", grads["dx"][b], *ref["dx"])
        if with_state:
            within("dstate0", grads["dstate0"][b], *ref["dstate0"])
        for name in ("dweight", "dbias"):
            v, e = sums.get(name, (0.0, 0.0))
            sums[name] = (v + ref[name][0], e + ref[name][1] + n * 2.0 ** -24 * ref[name][0].abs())
    within("dweight", grads["dweight"], *sums["dweight"])
    if with_bias:
        within("dbias", grads["dbias"], *sums["dbias"])


def test_packed_gradients_and_padding():
    gen = torch.Generator(device="cuda").manual_seed(3)
    lens, C, dtype = [5, 0, 70, 1, 2], 48, torch.float32
    cu, rows = _packed(lens, 19)
    x, dy = _normal(gen, rows, C), _normal(gen, rows, C)
    x[sum(lens):] = float("nan")  # padding may hold anything
    dy[sum(lens):] = float("nan")
    w, bias, s0, ds = _normal(gen, C, 4), _normal(gen, C), _normal(gen, 5, 3, C), _normal(gen, 5, 3, C)
    leaves = [t.requires_grad_() for t in (x, w, bias, s0)]
    y, state = gdn.causal_conv(*leaves, cu_seqlens=cu, flags=SILU)
    dx, dw, db, dst = torch.autograd.grad([y, state], leaves, [dy, ds])
    assert not bool(y[sum(lens):].any()) and not bool(dx[sum(lens):].any())
    vw, ew, vb, eb = 0, 0, 0, 0
    for b in range(5):
        r = slice(int(cu[b]), int(cu[b + 1]))
        ref = conv_seq(x[r], w, bias, s0[b], True, dy[r], ds[b])
        within("dx", dx[r], *ref["dx"])
        within("dstate0", dst[b], *ref["dstate0"])
        assert torch.equal(state[b].detach().double(), ref["state"][0])
        vw, ew, vb, eb = vw + ref["dweight"][0], ew + ref["dweight"][1], vb + ref["dbias"][0], eb + ref["dbias"][1]
    within("dweight", dw, vw, ew * 1.01)
    within("dbias", db, vb, eb * 1.01)


def test_differences():
    """Directional derivatives against central differences of the 64-bit form."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, w, b, s0 = (_normal(gen, *s) for s in ((2, 9, 8), (8, 3), (8,), (2, 2, 8)))
    dy, ds = _normal(gen, 2, 9, 8), _normal(gen, 2, 2, 8)

    def loss(x, w, b, s0):
        total = 0.0
        for i in range(2):
            seq = torch.cat((s0[i], x[i]))
            pre = sum(seq[j:j + 9] * w[:, j] for j in range(3)) + b
            total = total + (pre * torch.sigmoid(pre) * dy[i].double()).sum() + (seq[9:] * ds[i].double()).sum()
        return float(total)

    g = gdn.gdn_causal_conv_bwd(x, w, b, dy, state0=s0, dstate=ds, flags=SILU)
    args = [t.double() for t in (x, w, b, s0)]
    for i, name in enumerate(("dx", "dweight", "dbias", "dstate0")):
        v = torch.randn(args[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        up, down = (loss(*[a + s * 1e-5 * v if j == i else a for j, a in enumerate(args)]) for s in (1, -1))
        want = (up - down) / 2e-5
        got = float((g[name].double() * v).sum())
        # float32 products of a few hundred terms, and 1e-10 of curvature
        assert abs(got - want) <= 1e-5 * float((g[name].double().abs() * v.abs()).sum()) + 1e-7


def test_strided_rows_and_another_stream():
    gen = torch.Generator(device="cuda").manual_seed(5)
    qkv = _normal(gen, 2, 50, 3 * 64 + 8, dtype=torch.bfloat16)
    x, w = qkv[:, :, 64:128], _normal(gen, 64, 4, dtype=torch.bfloat16)
    want, _ = gdn.gdn_causal_conv_fwd(x.contiguous(), w, flags=SILU)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, _ = gdn.gdn_causal_conv_fwd(x, w, flags=SILU)
        odd, _ = gdn.gdn_causal_conv_fwd(qkv[:, :, 1:65], w, flags=SILU)  # not aligned to a vector
    side.synchronize()
    assert torch.equal(got, want)
    assert torch.equal(odd, gdn.gdn_causal_conv_fwd(qkv[:, :, 1:65].contiguous(), w, flags=SILU)[0])


def test_split_calls_carry_the_state():
    """The same tokens in one call and in pieces give the same bits."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    x, w = _normal(gen, 3, 41, 72, dtype=torch.bfloat16), _normal(gen, 72, 4, dtype=torch.bfloat16)
    whole, end = gdn.gdn_causal_conv_fwd(x, w, flags=SILU)
    state = torch.zeros(3, 3, 72, dtype=torch.bfloat16, device="cuda")
    parts, at = [], 0
    for n in (1, 2, 17, 1, 20):
        y, state = gdn.gdn_causal_conv_fwd(x[:, at:at + n].contiguous(), w, state0=state, state_final=state, flags=SILU)
        parts.append(y)
        at += n
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(state, end)


def test_captured_replay_with_other_lengths():
    gen = torch.Generator(device="cuda").manual_seed(7)
    C = 64
    x, w = _normal(gen, 24, C, dtype=torch.bfloat16), _normal(gen, C, 4, dtype=torch.bfloat16)
    cu = torch.tensor([0, 8, 24], dtype=torch.int32, device="cuda")
    kv = torch.tensor([8, 16], dtype=torch.int32, device="cuda")
    pool = torch.zeros(2, 3, C, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(x)

    def call():
        return gdn.gdn_causal_conv_fwd(x, w, state0=pool, state_final=pool, cu_seqlens=cu, kv_lens=kv, max_q=24, out=out, flags=SILU)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([8, 16], [1, 1], [0, 24], [20, 0]):
        cu.copy_(torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32))
        kv.copy_(torch.tensor(lens, dtype=torch.int32) + 3)
        pool.copy_(_normal(gen, 2, 3, C, dtype=torch.bfloat16))
        start = pool.clone()
        graph.replay()
        torch.cuda.synchronize()
        for b in range(2):
            r = slice(int(cu[b]), int(cu[b + 1]))
            ref = conv_seq(x[r], w, None, start[b], True)
            within("y", out[r], *ref["y"])
            assert torch.equal(pool[b].double(), ref["state"][0])


def test_bad_slots_are_reported():
    x, w = torch.ones(2, 8, device="cuda"), torch.ones(8, 4, device="cuda")
    pool = torch.ones(3, 3, 8, device="cuda")
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    y, _ = gdn.gdn_causal_conv_fwd(x, w, state0=pool, state_final=pool, cu_seqlens=cu, max_q=1,
                                   slots=torch.tensor([7, 1], dtype=torch.int32, device="cuda"))
    assert gdn.gdn_check_device_error() == gdn.binding.GDN_ERR_INTERNAL
    assert gdn.gdn_check_device_error() == 0
    assert bool((y[0] == 1).all()) and bool((y[1] == 4).all()) and bool((pool == 1).all())


def test_refusals():
    x, w = torch.zeros(2, 4, 8, device="cuda"), torch.zeros(8, 4, device="cuda")
    flat, cu = x.view(8, 8), torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    f = gdn.gdn_causal_conv_fwd
    bad = [lambda: f(flat, w), lambda: f(x[:, 1:], w), lambda: f(x, w, cu_seqlens=cu), lambda: f(x, w[:, :1]), lambda: f(x, torch.zeros(8, 5, device="cuda")),
           lambda: f(x, w[:4]), lambda: f(x.half(), w.half()), lambda: f(x, w.bfloat16()), lambda: f(x, w, torch.zeros(7, device="cuda")),
           lambda: f(x, w, state0=torch.zeros(1, 3, 8, device="cuda")), lambda: f(x, w, state0=torch.zeros(2, 2, 8, device="cuda")),
           lambda: f(flat, w, cu_seqlens=cu.long()), lambda: f(flat, w, cu_seqlens=cu, slots=slots, state0=torch.zeros(2, 3, 8, device="cuda")),
           lambda: f(flat, w, cu_seqlens=cu, slots=slots, state0=torch.zeros(2, 3, 8, device="cuda"), state_final=torch.zeros(3, 3, 8, device="cuda")),
           lambda: f(x, w.t().contiguous().t()), lambda: f(x.transpose(0, 1), w), lambda: f(flat, w, cu_seqlens=cu, max_q=0),
           lambda: f(x, w, flags=2), lambda: f(x, w, out=torch.zeros(1, 1, 8, device="cuda").expand(2, 4, 8)),
           lambda: f(x, w.clone().requires_grad_()), lambda: f(x.cpu(), w), lambda: f(x, w.cpu()), lambda: f(flat, w, cu_seqlens=cu.cpu())]
    for i, call in enumerate(bad):
        with pytest.raises(gdn.GdnError):
            call()
            pytest.fail(f"call {i} was not refused")
    y, state = gdn.causal_conv(x.requires_grad_(), w)
    (g,) = torch.autograd.grad(y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), x)


def test_empty_calls():
    w = torch.ones(8, 4, device="cuda")
    for shape in ((0, 5, 8), (3, 0, 8)):
        x = torch.zeros(*shape, device="cuda")
        s0 = torch.full((shape[0], 3, 8), 2.0, device="cuda")
        y, s = gdn.gdn_causal_conv_fwd(x, w, state0=s0)
        assert y.shape == x.shape and torch.equal(s, s0)
        g = gdn.gdn_causal_conv_bwd(x, w, None, x, state0=s0, dstate=s0)
        assert g["dx"].shape == x.shape and not bool(g["dweight"].any()) and torch.equal(g["dstate0"], s0)
