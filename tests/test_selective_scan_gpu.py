"""Selective scan against 64 bits: packed and batched, states in pools, split and whole sequences, gradients, refusals."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn
from tests.mixer_reference import over_channels, scan_seq, within

pytestmark = pytest.mark.gpu
SOFT = gdn.GDN_FLAG_DT_SOFTPLUS


def _normal(gen, *shape, dtype=torch.float32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)


def _inputs(gen, lead, D, G, S, dtype, gate, extra):
    """Inputs as a model has them: B and C views of one projection; extra: skip and bias."""
    bc = _normal(gen, *lead, 2 * G * S, dtype=dtype)
    B, C = (t.unflatten(-1, (G, S)) for t in bc.split(G * S, -1))
    A = -torch.arange(1, S + 1, device="cuda") * torch.exp(_normal(gen, D, S, std=0.2))
    return dict(u=_normal(gen, *lead, D, dtype=dtype), dt=_normal(gen, *lead, D, dtype=dtype, std=0.7), A=A, B=B, C=C,
                D=_normal(gen, D) if extra else None, z=_normal(gen, *lead, D, dtype=dtype) if gate else None,
                dt_bias=_normal(gen, D, mean=-3.0) if extra else None)


def _rows(s, r, **more):
    """The reference's arguments for a sequence's rows."""
    cut = {k: s[k][r] for k in ("u", "dt", "B", "C")}
    return dict(cut, A=s["A"], D=s["D"], z=None if s["z"] is None else s["z"][r], bias=s["dt_bias"], **more)


# lengths, rows behind, channels, groups, states, gate, skip and bias, softplus
PACKED = [([1] * 4, 0, 768, 1, 16, True, True, True), ([1, 2, 3, 4, 5], 3, 64, 1, 16, True, True, True),
          ([0, 7, 0, 1, 0], 9, 40, 2, 8, False, True, True), ([33, 129, 1], 70, 37, 1, 16, True, False, True),
          ([300, 17], 1, 100, 4, 32, True, True, True), ([1], 0, 1, 1, 16, True, True, True), ([64, 16, 65], 0, 30, 3, 64, False, True, True),
          ([], 20, 16, 1, 16, True, True, True), ([15, 16, 17], 40, 132, 1, 16, True, True, True), ([9, 8, 7], 2, 72, 1, 8, True, True, True),
          ([1, 0, 1, 1, 1] * 13, 3, 404, 1, 64, True, True, True), ([1] * 66, 0, 410, 2, 64, False, False, True)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,pad,D,G,S,gate,extra,soft", PACKED)
def test_packed_forward(lens, pad, D, G, S, gate, extra, soft, dtype):
    gen = torch.Generator(device="cuda").manual_seed(sum(lens) * 7 + D)
    n, pool, rows = len(lens), len(lens) + 4, sum(lens) + pad
    cu = torch.tensor([sum(lens[:b]) for b in range(n + 1)], dtype=torch.int32, device="cuda")
    s = _inputs(gen, (rows,), D, G, S, dtype, gate, extra)
    states = _normal(gen, pool, D, S)
    slots = torch.randperm(pool, generator=gen, device="cuda")[:n].to(torch.int32)
    if n > 2:
        slots[1] = -1
    past = [0 if b == n - 1 and n > 1 else 5 for b in range(n)]
    kv = torch.tensor([p + v for p, v in zip(past, lens)], dtype=torch.int32, device="cuda")
    after = torch.full((pool, D, S), 3.0, device="cuda")
    call = dict(slots=slots, cu_seqlens=cu, kv_lens=kv, max_q=max(lens + [1]), flags=SOFT if soft else 0)
    y, got, kept = gdn.gdn_selective_scan_fwd(**s, h0=states, h_final=after, **call)
    assert got is after and kept is None
    written = set()
    for b in range(n):
        slot = int(slots[b])
        h0 = states[slot] if slot >= 0 and past[b] > 0 else None
        ref = scan_seq(**_rows(s, slice(int(cu[b]), int(cu[b + 1])), softplus=soft, h0=h0))
        within("y", y[int(cu[b]):int(cu[b + 1])], *ref["y"])
        if slot >= 0:
            within("h", after[slot], *ref["h"])
            written.add(slot)
    for slot in set(range(pool)) - written:
        assert bool((after[slot] == 3).all())
    assert not bool(y[sum(lens):].any())
    # in place, and into given rows with gaps: the rows behind the last sequence are left alone
    wide, own = torch.full((rows, D + 8), 7.0, dtype=dtype, device="cuda"), states.clone()
    y2, _, _ = gdn.gdn_selective_scan_fwd(**s, h0=own, h_final=own, out=wide[:, :D], **call)
    assert torch.equal(y2[:sum(lens)], y[:sum(lens)]) and bool((wide[sum(lens):] == 7).all()) and bool((wide[:, D:] == 7).all())
    for slot in range(pool):
        assert torch.equal(own[slot], after[slot] if slot in written else states[slot])
    assert gdn.gdn_check_device_error() == 0


# sequences, tokens, channels, groups, states, gate, skip and bias, softplus, state, gradient of the last state
TRAIN = [(2, 40, 96, 1, 16, True, True, True, False, False), (3, 17, 37, 1, 16, True, True, True, True, True),
         (1, 1, 64, 1, 16, True, True, True, True, True), (2, 33, 30, 3, 8, False, True, True, True, False),
         (1, 700, 24, 1, 16, True, True, True, True, True), (2, 50, 72, 2, 64, True, True, True, False, True),
         (2, 21, 136, 1, 32, False, False, True, True, True), (1, 19, 260, 1, 16, True, True, False, True, True),
         (1, 9, 1040, 1, 64, True, True, True, True, True), (2, 5, 2052, 2, 64, False, True, True, False, False),
         (3, 900, 5, 1, 8, True, True, True, True, True)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,T,D,G,S,gate,extra,soft,with_h0,with_dh", TRAIN)
def test_training(n, T, D, G, S, gate, extra, soft, with_h0, with_dh, dtype):
    gen = torch.Generator(device="cuda").manual_seed(n * T + D)
    s = _inputs(gen, (n, T), D, G, S, dtype, gate, extra)
    if not soft:
        s["dt"] = s["dt"].abs() * 0.1  # steps themselves
        s["dt_bias"] = s["dt_bias"].abs() * 0.01
    h0 = _normal(gen, n, D, S) if with_h0 else None
    dy, dh = _normal(gen, n, T, D, dtype=dtype), _normal(gen, n, D, S) if with_dh else None
    named = dict(s, h0=h0)
    leaves = {k: t.requires_grad_() for k, t in named.items() if t is not None}
    y, h = gdn.selective_scan(*[named[k] for k in ("u", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0")], flags=SOFT if soft else 0)
    outs, gs = ([y, h], [dy, dh]) if with_dh else ([y], [dy])
    got = dict(zip(leaves, torch.autograd.grad(outs, list(leaves.values()), gs)))
    s = {k: None if t is None else t.detach() for k, t in s.items()}
    sums = {}
    for b in range(n):
        ref = scan_seq(**_rows(s, b, softplus=soft, h0=None if h0 is None else h0[b].detach(), dy=dy[b], dh=None if dh is None else dh[b]))
        within("y", y[b].detach(), *ref["y"])
        within("h", h[b].detach(), *ref["h"])
        within("du", got["u"][b], *ref["du"])
        within("ddt", got["dt"][b], *ref["ddt"])
        within("dB", got["B"][b], *over_channels(ref["dB"], G))
        within("dC", got["C"][b], *over_channels(ref["dC"], G))
        if gate:
            within("dz", got["z"][b], *ref["dz"])
        if with_h0:
            within("dh0", got["h0"][b], *ref["dh0"])
        for name in ("dA", "dD", "ddt_bias"):
            v, e = sums.get(name, (0.0, 0.0))
            sums[name] = (v + ref[name][0], e + ref[name][1] + n * 2.0 ** -24 * ref[name][0].abs())
    within("dA", got["A"], *sums["dA"])
    if extra:
        within("dD", got["D"], *sums["dD"])
        within("ddt_bias", got["dt_bias"], *sums["ddt_bias"])


def test_packed_gradients_and_padding():
    gen = torch.Generator(device="cuda").manual_seed(3)
    lens, D, S = [5, 0, 70, 1, 2], 48, 16
    rows = sum(lens) + 19
    cu = torch.tensor([sum(lens[:b]) for b in range(6)], dtype=torch.int32, device="cuda")
    s = _inputs(gen, (rows,), D, 1, S, torch.float32, True, True)
    for k in ("u", "dt", "B", "C", "z"):
        s[k][sum(lens):] = float("nan")  # padding may hold anything
    h0, dh, dy = _normal(gen, 5, D, S), _normal(gen, 5, D, S), _normal(gen, rows, D)
    dy[sum(lens):] = float("nan")
    y, h, kept = gdn.gdn_selective_scan_fwd(**s, h0=h0, cu_seqlens=cu, flags=SOFT, save=True)
    g = gdn.gdn_selective_scan_bwd(s["u"], s["dt"], s["A"], s["B"], s["C"], dy, kept, D=s["D"], z=s["z"], dt_bias=s["dt_bias"], dh_final=dh,
                                   need_dh0=True, cu_seqlens=cu, flags=SOFT)
    for t in (y, g["du"], g["ddt"], g["dz"], g["dB"], g["dC"]):
        assert not bool(t[sum(lens):].any())
    sums = {}
    for b in range(5):
        r = slice(int(cu[b]), int(cu[b + 1]))
        ref = scan_seq(**_rows(s, r, h0=h0[b], dy=dy[r], dh=dh[b]))
        for name, t in (("y", y[r]), ("h", h[b]), ("du", g["du"][r]), ("ddt", g["ddt"][r]), ("dz", g["dz"][r]), ("dh0", g["dh0"][b])):
            within(name, t, *ref[name])
        within("dB", g["dB"][r], *over_channels(ref["dB"], 1))
        within("dC", g["dC"][r], *over_channels(ref["dC"], 1))
        for name in ("dA", "dD", "ddt_bias"):
            v, e = sums.get(name, (0.0, 0.0))
            sums[name] = (v + ref[name][0], (e + ref[name][1]) * 1.01)
    for name in ("dA", "dD", "ddt_bias"):
        within(name, g[name], *sums[name])


@pytest.mark.parametrize("S,D,G,T", [(16, 32, 1, 3000), (64, 16, 2, 1500), (8, 72, 1, 2500), (32, 20, 1, 2100)])
def test_long_sequences_in_chunks(S, D, G, T):
    """Few channels and many tokens: sequences are split, forward and backward; a ragged batch and empty sequences too."""
    gen = torch.Generator(device="cuda").manual_seed(S + T)
    lens = [T, 0, 1, T // 3]
    rows = sum(lens) + 5
    cu = torch.tensor([sum(lens[:b]) for b in range(5)], dtype=torch.int32, device="cuda")
    s = _inputs(gen, (rows,), D, G, S, torch.float32, True, True)
    dims = gdn.binding.GdnScanDims(D, G, S, gdn.GDN_F32, SOFT)
    seqs = gdn.binding.GdnPacked(rows, 4, 4, 1 << 20, None, None)
    lib = gdn.load()
    assert lib.gdn_selective_scan_workspace_bytes(dims, seqs, T) > 0  # the forward splits
    h0, dh, dy = _normal(gen, 4, D, S), _normal(gen, 4, D, S), _normal(gen, rows, D)
    y, h, kept = gdn.gdn_selective_scan_fwd(**s, h0=h0, cu_seqlens=cu, max_q=T, flags=SOFT, save=True)
    g = gdn.gdn_selective_scan_bwd(s["u"], s["dt"], s["A"], s["B"], s["C"], dy, kept, D=s["D"], z=s["z"], dt_bias=s["dt_bias"], dh_final=dh,
                                   need_dh0=True, cu_seqlens=cu, max_q=T, flags=SOFT)
    sums = {}
    for b in range(4):
        r = slice(int(cu[b]), int(cu[b + 1]))
        ref = scan_seq(**_rows(s, r, h0=h0[b], dy=dy[r], dh=dh[b]))
        for name, t in (("y", y[r]), ("h", h[b]), ("du", g["du"][r]), ("ddt", g["ddt"][r]), ("dz", g["dz"][r]), ("dh0", g["dh0"][b])):
            within(name, t, *ref[name])
        within("dB", g["dB"][r], *over_channels(ref["dB"], G))
        within("dC", g["dC"][r], *over_channels(ref["dC"], G))
        for name in ("dA", "dD", "ddt_bias"):
            v, e = sums.get(name, (0.0, 0.0))
            sums[name] = (v + ref[name][0], (e + ref[name][1]) * 1.01)
    for name in ("dA", "dD", "ddt_bias"):
        within(name, g[name], *sums[name])


def test_differences():
    """Directional derivatives against central differences of the 64-bit form."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    s = _inputs(gen, (1, 9), 8, 2, 8, torch.float32, True, True)
    h0, dy, dh = _normal(gen, 1, 8, 8), _normal(gen, 1, 9, 8), _normal(gen, 1, 8, 8)
    _, _, kept = gdn.gdn_selective_scan_fwd(**s, h0=h0, flags=SOFT, save=True)
    g = gdn.gdn_selective_scan_bwd(s["u"], s["dt"], s["A"], s["B"], s["C"], dy, kept, D=s["D"], z=s["z"], dt_bias=s["dt_bias"], dh_final=dh,
                                   need_dh0=True, flags=SOFT)
    args = {k: t.double() for k, t in dict(s, h0=h0).items()}

    def loss(a):
        ref = scan_seq(a["u"][0], a["dt"][0], a["A"], a["B"][0], a["C"][0], a["D"], a["z"][0], a["dt_bias"], True, a["h0"][0])
        return float((ref["y"][0] * dy[0].double()).sum() + (ref["h"][0] * dh[0].double()).sum())

    for k, a in args.items():
        v = torch.randn(a.shape, generator=gen, device="cuda", dtype=torch.float64)
        up, down = (loss(dict(args, **{k: a + sign * 1e-5 * v})) for sign in (1, -1))
        got, want = float((g["d" + k].double() * v).sum()), (up - down) / 2e-5
        # float32 over a few hundred terms, and 1e-10 of curvature
        assert abs(got - want) <= 2e-5 * float((g["d" + k].double().abs() * v.abs()).sum()) + 1e-6, k


@pytest.mark.parametrize("S,D,dtype", [(16, 20, torch.float32), (8, 36, torch.bfloat16), (64, 12, torch.bfloat16)])
def test_states_in_a_pool_over_many_chunks(S, D, dtype):
    """Hundreds of short chunks a sequence beside empty and short ones; states read and written in place."""
    gen = torch.Generator(device="cuda").manual_seed(40 + S)
    lens, past, slots = [1700, 0, 40, 1, 521], [3, 5, 0, 2, 0], [4, 0, 6, 2, -1]
    rows = sum(lens)
    cu = torch.tensor([sum(lens[:b]) for b in range(6)], dtype=torch.int32, device="cuda")
    kv = torch.tensor([p + n for p, n in zip(past, lens)], dtype=torch.int32, device="cuda")
    s = _inputs(gen, (rows,), D, 1, S, dtype, True, True)
    s["dt_bias"] -= 2.0  # states that outlive chunks
    states = _normal(gen, 7, D, S)
    own = states.clone()
    y, _, _ = gdn.gdn_selective_scan_fwd(**s, h0=own, h_final=own, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"),
                                         cu_seqlens=cu, kv_lens=kv, max_q=1700, flags=SOFT)
    for b, slot in enumerate(slots):
        r = slice(int(cu[b]), int(cu[b + 1]))
        ref = scan_seq(**_rows(s, r, h0=states[slot] if slot >= 0 and past[b] else None))
        within("y", y[r], *ref["y"])
        if slot >= 0:
            within("h", own[slot], *ref["h"])
    for slot in set(range(7)) - set(slots):
        assert torch.equal(own[slot], states[slot])
    assert gdn.gdn_check_device_error() == 0


@pytest.mark.parametrize("n", [70, 71])
def test_single_tokens_of_a_batch(n):
    """More channels and sequences than one of each a warp would fit; an odd and an even number of them."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    s = _inputs(gen, (n, 1), 400, 1, 64, torch.bfloat16, True, True)
    h0 = _normal(gen, n, 400, 64)
    own = h0.clone()
    y, h, _ = gdn.gdn_selective_scan_fwd(**s, h0=own, h_final=own, flags=SOFT)
    for b in range(n):
        ref = scan_seq(**_rows(s, b, h0=h0[b]))
        within("y", y[b], *ref["y"])
        within("h", h[b], *ref["h"])


def test_split_calls_carry_the_state():
    gen = torch.Generator(device="cuda").manual_seed(6)
    s = _inputs(gen, (2, 60), 40, 1, 16, torch.float32, True, True)
    whole, end, _ = gdn.gdn_selective_scan_fwd(**s, flags=SOFT)
    state, parts, at = torch.zeros(2, 40, 16, device="cuda"), [], 0
    for n in (1, 17, 1, 40, 1):
        cut = {k: (t[:, at:at + n].contiguous() if k in ("u", "dt", "B", "C", "z") else t) for k, t in s.items()}
        y, state, _ = gdn.gdn_selective_scan_fwd(**cut, h0=state, h_final=state, flags=SOFT)
        parts.append(y)
        at += n
    for b in range(2):
        ref = scan_seq(**_rows(s, b))
        within("y", torch.cat(parts, 1)[b], *ref["y"])
        within("h", state[b], *ref["h"])
        within("y", whole[b], *ref["y"])
        within("h", end[b], *ref["h"])


def test_same_bits_every_time_and_on_another_stream():
    gen = torch.Generator(device="cuda").manual_seed(8)
    s = _inputs(gen, (2, 600), 200, 1, 16, torch.bfloat16, True, True)
    dy = _normal(gen, 2, 600, 200, dtype=torch.bfloat16)

    def step():
        y, h, kept = gdn.gdn_selective_scan_fwd(**s, flags=SOFT, save=True)
        g = gdn.gdn_selective_scan_bwd(s["u"], s["dt"], s["A"], s["B"], s["C"], dy, kept, D=s["D"], z=s["z"], dt_bias=s["dt_bias"], flags=SOFT)
        return [y, h] + [t for t in g.values() if t is not None]

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = step()
    third = step()
    side.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_captured_training_step_replays():
    gen = torch.Generator(device="cuda").manual_seed(9)
    s = _inputs(gen, (1, 300), 64, 1, 16, torch.float32, True, True)
    dy = _normal(gen, 1, 300, 64)

    def step():
        y, h, kept = gdn.gdn_selective_scan_fwd(**s, flags=SOFT, save=True)
        g = gdn.gdn_selective_scan_bwd(s["u"], s["dt"], s["A"], s["B"], s["C"], dy, kept, D=s["D"], z=s["z"], dt_bias=s["dt_bias"], flags=SOFT)
        return [y, h] + [t for t in g.values() if t is not None]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(2):
        s["u"].copy_(_normal(gen, 1, 300, 64))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b)


def test_nonfinite_values_stay_in_their_channel():
    gen = torch.Generator(device="cuda").manual_seed(10)
    s = _inputs(gen, (1, 40), 70, 1, 16, torch.float32, False, True)
    s["u"][0, 11, 33] = float("nan")
    y, h, _ = gdn.gdn_selective_scan_fwd(**s, flags=SOFT)
    bad = torch.isnan(y[0])
    assert bool(bad[11:, 33].all()) and int(bad.sum()) == 29 and bool(torch.isnan(h[0, 33]).all()) and int(torch.isnan(h).sum()) == 16


def test_wide_steps():
    """Steps from vanishing to long ones: softplus keeps its precision at both ends."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    s = _inputs(gen, (1, 64), 32, 1, 16, torch.float32, False, False)
    s["dt"] = torch.linspace(-40, 40, 64 * 32, device="cuda").view(1, 64, 32).contiguous()
    y, h, _ = gdn.gdn_selective_scan_fwd(**s, flags=SOFT)
    ref = scan_seq(**_rows(s, 0))
    within("y", y[0], *ref["y"])
    within("h", h[0], *ref["h"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,G,S", [(768, 1, 16), (50, 2, 8), (37, 1, 16), (96, 1, 64), (24, 1, 32)])
def test_single_tokens(D, G, S, dtype):
    """No token, one or two a sequence, some without a state; and the same call whose bound says fewer than there are."""
    gen = torch.Generator(device="cuda").manual_seed(D + S)
    lens = [1, 0, 2, 1, 2, 0]
    cu = torch.tensor([sum(lens[:b]) for b in range(7)], dtype=torch.int32, device="cuda")
    s = _inputs(gen, (sum(lens) + 2,), D, G, S, dtype, True, True)
    states, slots = _normal(gen, 9, D, S), torch.tensor([3, 5, -1, 0, 8, 2], dtype=torch.int32, device="cuda")
    kv = torch.tensor([v + p for v, p in zip(lens, [4, 4, 4, 0, 4, 0])], dtype=torch.int32, device="cuda")
    for bound in (2, 1):
        after = torch.full_like(states, 3.0)
        y, _, _ = gdn.gdn_selective_scan_fwd(**s, h0=states, h_final=after, slots=slots, cu_seqlens=cu, kv_lens=kv, max_q=bound, flags=SOFT)
        for b in range(6):
            slot, r = int(slots[b]), slice(int(cu[b]), int(cu[b + 1]))
            ref = scan_seq(**_rows(s, r, h0=states[slot] if slot >= 0 and b not in (3, 5) else None))
            within("y", y[r], *ref["y"])
            if slot >= 0:
                within("h", after[slot], *ref["h"])
        assert not bool(y[sum(lens):].any()) and bool((after[[1, 4, 6, 7]] == 3).all())


def test_bounds_choose_no_result():
    """max_q below, at and far above the longest sequence: the same within float32."""
    gen = torch.Generator(device="cuda").manual_seed(21)
    lens = [700, 3, 0, 90]
    cu = torch.tensor([sum(lens[:b]) for b in range(5)], dtype=torch.int32, device="cuda")
    s = _inputs(gen, (sum(lens),), 32, 1, 16, torch.float32, True, True)
    dy = _normal(gen, sum(lens), 32)
    for bound in (1, 5, 700, None, 2 ** 31 - 1):
        y, h, kept = gdn.gdn_selective_scan_fwd(**s, cu_seqlens=cu, max_q=bound, flags=SOFT, save=True)
        g = gdn.gdn_selective_scan_bwd(s["u"], s["dt"], s["A"], s["B"], s["C"], dy, kept, D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                                       cu_seqlens=cu, max_q=bound, flags=SOFT)
        for b in range(4):
            r = slice(int(cu[b]), int(cu[b + 1]))
            ref = scan_seq(**_rows(s, r, dy=dy[r]))
            for name, t in (("y", y[r]), ("h", h[b]), ("du", g["du"][r]), ("ddt", g["ddt"][r]), ("dz", g["dz"][r])):
                within(name, t, *ref[name])


def test_strides_beyond_32_bits():
    """Rows more than 2^31 elements apart."""
    gen = torch.Generator(device="cuda").manual_seed(22)
    s = _inputs(gen, (1, 3), 8, 1, 16, torch.bfloat16, True, True)
    far = torch.empty(2 * (2 ** 31 + 64) + 64, dtype=torch.bfloat16, device="cuda")
    u = far.as_strided((1, 3, 8), (3 * (2 ** 31 + 64), 2 ** 31 + 64, 1))
    u.copy_(s["u"])
    dy = _normal(gen, 1, 3, 8, dtype=torch.bfloat16)
    res = []
    for x in (s["u"], u):
        y, h, kept = gdn.gdn_selective_scan_fwd(**dict(s, u=x), flags=SOFT, save=True)
        g = gdn.gdn_selective_scan_bwd(x, s["dt"], s["A"], s["B"], s["C"], dy, kept, D=s["D"], z=s["z"], dt_bias=s["dt_bias"], flags=SOFT)
        w = torch.ones(8, 4, dtype=torch.bfloat16, device="cuda")
        c, _ = gdn.gdn_causal_conv_fwd(x, w)
        res.append([y, h, c, gdn.gdn_causal_conv_bwd(x, w, None, dy)["dweight"]] + [t for t in g.values() if t is not None])
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_only_padding():
    """No sequences at all, and rows of padding enough for a split."""
    gen = torch.Generator(device="cuda").manual_seed(24)
    s = _inputs(gen, (5000,), 32, 1, 16, torch.float32, True, True)
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, h, kept = gdn.gdn_selective_scan_fwd(**s, cu_seqlens=cu, flags=SOFT, save=True)
    g = gdn.gdn_selective_scan_bwd(s["u"], s["dt"], s["A"], s["B"], s["C"], s["u"], kept, D=s["D"], z=s["z"], dt_bias=s["dt_bias"], cu_seqlens=cu, flags=SOFT)
    assert h.shape == (0, 32, 16) and not bool(y.any()) and not any(bool(t.any()) for t in g.values() if t is not None)


def test_growing_states_without_inputs():
    """A above zero: factors over a chunk overflow, and a channel without inputs stays zero all the same."""
    gen = torch.Generator(device="cuda").manual_seed(25)
    s = _inputs(gen, (1, 4000), 32, 1, 16, torch.float32, False, False)
    s["A"], s["dt"] = torch.full_like(s["A"], 0.5), torch.full_like(s["dt"], 1.0)
    s["u"].zero_()
    y, h, kept = gdn.gdn_selective_scan_fwd(**s, flags=SOFT, save=True)
    assert not bool(y.any()) and not bool(h.any())
    g = gdn.gdn_selective_scan_bwd(s["u"], s["dt"], s["A"], s["B"], s["C"], torch.zeros_like(y), kept, flags=SOFT)
    assert not any(bool(t.any()) for t in g.values() if t is not None)


def test_two_calls_at_once():
    """Calls on two streams with workspaces of their own give what they give one after the other."""
    gen = torch.Generator(device="cuda").manual_seed(23)
    sets = [_inputs(gen, (1, 2000), 64, 1, 16, torch.float32, True, True) for _ in range(2)]
    dys = [_normal(gen, 1, 2000, 64) for _ in range(2)]

    def step(s, dy):
        y, h, kept = gdn.gdn_selective_scan_fwd(**s, flags=SOFT, save=True)
        g = gdn.gdn_selective_scan_bwd(s["u"], s["dt"], s["A"], s["B"], s["C"], dy, kept, D=s["D"], z=s["z"], dt_bias=s["dt_bias"], flags=SOFT)
        return [y, h] + [t for t in g.values() if t is not None]

    alone = [step(s, dy) for s, dy in zip(sets, dys)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    together = [[], []]
    for _ in range(3):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                together[i].append(step(sets[i], dys[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for got in together[i]:
            for a, b in zip(alone[i], got):
                assert torch.equal(a, b)


def test_refusals():
    gen = torch.Generator(device="cuda").manual_seed(12)
    s = _inputs(gen, (2, 4), 8, 1, 16, torch.float32, True, True)
    flat = {k: (t.flatten(0, 1) if k in ("u", "dt", "B", "C", "z") else t) for k, t in s.items()}
    cu = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    h0 = torch.zeros(2, 8, 16, device="cuda")
    f = gdn.gdn_selective_scan_fwd
    bad = [lambda: f(**flat), lambda: f(**s, cu_seqlens=cu), lambda: f(**dict(s, A=s["A"][:, :12].contiguous())), lambda: f(**dict(s, A=s["A"].bfloat16())),
           lambda: f(**dict(s, dt=s["dt"].bfloat16())), lambda: f(**dict(s, B=s["B"][..., :8])), lambda: f(**dict(s, C=s["C"][:, :3])),
           lambda: f(**dict(s, B=s["B"].repeat(1, 1, 3, 1), C=s["C"].repeat(1, 1, 3, 1))), lambda: f(**dict(s, D=s["D"][:4])),
           lambda: f(**s, h0=h0[:1]), lambda: f(**s, h0=h0.bfloat16()), lambda: f(**flat, cu_seqlens=cu, slots=slots, h0=h0),
           lambda: f(**flat, cu_seqlens=cu, slots=slots, h0=h0, h_final=h0, save=True), lambda: f(**flat, cu_seqlens=cu, max_q=0),
           lambda: f(**s, flags=1), lambda: f(**dict(s, z=s["z"].cpu())), lambda: f(**dict(s, A=s["A"].clone().requires_grad_())),
           lambda: f(**s, out=torch.zeros(1, 1, 8, device="cuda").expand(2, 4, 8)),
           lambda: gdn.gdn_selective_scan_bwd(s["u"], s["dt"], s["A"], s["B"], s["C"], s["u"], torch.zeros(4, device="cuda"), flags=SOFT)]
    for i, call in enumerate(bad):
        with pytest.raises(gdn.GdnError):
            call()
            pytest.fail(f"call {i} was not refused")


def test_empty_calls():
    gen = torch.Generator(device="cuda").manual_seed(13)
    for lead in ((0, 5), (3, 0)):
        s = _inputs(gen, lead, 8, 1, 16, torch.float32, True, True)
        h0 = torch.full((lead[0], 8, 16), 2.0, device="cuda")
        y, h, kept = gdn.gdn_selective_scan_fwd(**s, h0=h0, flags=SOFT, save=True)
        assert y.shape == s["u"].shape and torch.equal(h, h0)
        g = gdn.gdn_selective_scan_bwd(s["u"], s["dt"], s["A"], s["B"], s["C"], s["u"], kept, D=s["D"], z=s["z"], dt_bias=s["dt_bias"], dh_final=h0,
                                       need_dh0=True, flags=SOFT)
        assert torch.equal(g["dh0"], h0) and not any(bool(g[k].any()) for k in ("dA", "dD", "ddt_bias"))
