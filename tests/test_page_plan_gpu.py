"""The plan of a serving step against lists: mixed steps, scarce pages, odd lengths, refusals, and a run with the calls that
read it."""
import random

import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn
from tests.mixer_reference import plan

pytestmark = pytest.mark.gpu


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _case(rng, n, page, cap, free, kind):
    """Requests with pages of their own from one shuffled pool."""
    pool = list(range(n * cap + free))
    rng.shuffle(pool)
    lens = [rng.choice([0, 1, page, page - 1, rng.randint(0, cap * page)]) for _ in range(n)]
    lens = [min(v, cap * page) for v in lens]
    table = []
    for v in lens:
        used = -(-v // page)
        table.append([pool.pop() for _ in range(used)] + [-1] * (cap - used))
    stack = [pool.pop() for _ in range(min(free, len(pool)))]
    new = []
    for v in lens:
        new.append({"step": 1, "idle": 0}.get(kind, rng.choice([0, 1, 1, 2, -1, -3, -v, -10 ** 6, rng.randint(1, 2 * page), rng.randint(0, cap * page)])))
    return table, lens, new, stack + [-7] * (n * cap), len(stack)


def _check(table, lens, new, free, count, page, top, error=False):
    t, f = _int(table).view(len(lens), -1), _int(free)
    got = gdn.gdn_page_plan(t, _int(lens), _int(new), f, _int([count]), page_size=page, max_tokens=top)
    want = plan(table, lens, new, free, count, page, top)
    for k, v in want.items():
        have = {"page_table": t, "free_pages": f}.get(k, getattr(got, k, None)).tolist()
        assert have == v, k
    bad = gdn.gdn_check_device_error()
    assert (bad != 0) == error
    return got


@pytest.mark.parametrize("kind", ["step", "idle", "mixed", "mixed"])
@pytest.mark.parametrize("n,page,cap,free,top", [(1, 16, 4, 3, 40), (5, 1, 9, 4, 30), (37, 16, 8, 20, 900), (300, 48, 5, 1000, 40000),
                                                 (700, 64, 3, 0, 700), (1025, 16, 4, 333, 2000), (64, 256, 2, 500, 1)])
def test_against_lists(n, page, cap, free, top, kind):
    rng = random.Random(n * 31 + page + len(kind))
    table, lens, new, stack, count = _case(rng, n, page, cap, free, kind)
    full = any(v > 0 and length + v > cap * page for length, v in zip(lens, new))
    _check(table, lens, new, stack, count, page, top, error=full)


def test_many_requests():
    rng = random.Random(5)
    table, lens, new, stack, count = _case(rng, 8192, 16, 2, 3000, "step")
    full = any(length + 1 > 32 for length in lens)
    _check(table, lens, new, stack, count, 16, 9000, error=full)


def test_pages_run_out_in_order():
    # three pages: the first and third get theirs, the fourth needs none, the second is left out
    got = _check([[-1] * 4, [-1] * 4, [-1] * 4, [9, -1, -1, -1]], [0, 0, 0, 3], [16, 64, 16, 1], [4, 5, 6, -1], 3, 16, 200)
    assert got.cu_seqlens.tolist() == [0, 16, 16, 16, 17]  # the third asks behind the second, which asks for more than there is
    assert got.free_count.tolist() == [2]


def test_pages_given_back_are_taken_in_the_same_step():
    got = _check([[3, 4, 5], [-1] * 3], [48, 0], [-48, 40], [-1] * 8, 0, 16, 64)
    assert got.slots.tolist()[:2] == [5 * 16, 5 * 16 + 1] and got.free_count.tolist() == [0]


def test_bad_values_are_reported():
    _check([[1, 2]], [33], [1], [7, -1], 1, 16, 8, error=True)  # clamped to the row, which is full then
    _check([[1, 2]], [-5], [1], [7, -1], 1, 16, 8, error=True)
    _check([[1, 2]], [20], [-20], [7], 1, 16, 8, error=True)  # the stack overflows
    _check([[1, 2]], [2 ** 31 - 1], [2 ** 31 - 1], [7], 1, 16, 8, error=True)


def test_large_slots_and_no_requests():
    big = 2 ** 27 + 3
    got = gdn.gdn_page_plan(
        _int([[big, -1]]), _int([5]), _int([2]), _int([0]), _int([0]), page_size=64, max_tokens=3)
    assert got.slots.tolist() == [big * 64 + 5, big * 64 + 6, -1]
    empty = gdn.gdn_page_plan(torch.empty(0, 4, dtype=torch.int32, device="cuda"), _int([]), _int([]), _int([1, 2]), _int([2]), page_size=16, max_tokens=5)
    assert empty.cu_seqlens.tolist() == [0] and empty.free_count.tolist() == [2] and empty.slots.tolist() == [-1] * 5


def test_captured_steps():
    """A captured plan replays with the lengths and the stack that are there."""
    table, stack = _int([[-1] * 8] * 3), _int(list(range(24)))
    lens, new, count = _int([0, 0, 0]), _int([20, 1, 0]), _int([24])

    def call():
        p = gdn.gdn_page_plan(table, lens, new, stack, count, page_size=16, max_tokens=64)
        lens.copy_(p.kv_lens)
        count.copy_(p.free_count)
        return p

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            p = call()
    torch.cuda.synchronize()
    state = plan([[-1] * 8] * 3, [0, 0, 0], [20, 1, 0], list(range(24)), 24, 16, 64)
    for step in ([20, 1, 0], [1, 1, 40], [-30, 1, 1], [5, -50, 30]):
        new.copy_(_int(step))
        held = (table.tolist(), lens.tolist(), step, stack.tolist(), int(count))
        graph.replay()
        torch.cuda.synchronize()
        want = plan(*held, 16, 64)
        for k in ("cu_seqlens", "requests", "positions", "slots"):
            assert getattr(p, k).tolist() == want[k], k
        assert lens.tolist() == want["kv_lens"] and count.tolist() == want["free_count"] and table.tolist() == want["page_table"]
    assert state["free_count"] == [21]


def test_refusals():
    t, v, f, c = _int([[1, 2]]), _int([0]), _int([3]), _int([1])
    g = gdn.gdn_page_plan
    bad = [lambda: g(t.long(), v, v, f, c, page_size=16, max_tokens=4), lambda: g(t, _int([0, 0]), v, f, c, page_size=16, max_tokens=4),
           lambda: g(t, v, v, f, _int([1, 2]), page_size=16, max_tokens=4), lambda: g(t, v, v, f, c, page_size=0, max_tokens=4),
           lambda: g(t, v, v, f, c, page_size=16, max_tokens=-1), lambda: g(t, v, v, f, c, page_size=16, max_tokens=2 ** 31),
           lambda: g(t.cpu(), v, v, f, c, page_size=16, max_tokens=4), lambda: g(t, v, v, f.cpu(), c, page_size=16, max_tokens=4),
           lambda: g(t.t(), v, v, f, c, page_size=16, max_tokens=4), lambda: g(_int([[1]] * 8193), _int([0] * 8193), _int([0] * 8193), f, c, page_size=16, max_tokens=4)]
    for i, call in enumerate(bad):
        with pytest.raises(gdn.GdnError):
            call()
            pytest.fail(f"call {i} was not refused")


def test_a_step_through_cache_attention_convolution_and_scan():
    """Three requests served as the plan says, steps of prompts and single tokens, one rolled back, against each request alone:
    the paged cache with its attention, the convolution and the scan all read the plan's arrays."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    R, page, cap, D, S, H, W = 3, 16, 6, 64, 16, 2, 64
    total = [50, 37, 70]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    data = [dict(x=normal(n, D), dt=normal(n, D), B=normal(n, 1, S), C=normal(n, 1, S), q=normal(n, H, W), k=normal(n, H, W), v=normal(n, H, W)) for n in total]
    weight, A = normal(D, 4), -torch.rand(D, S, generator=gen, device="cuda") * 4
    flags = dict(conv=gdn.GDN_FLAG_CONV_SILU, scan=gdn.GDN_FLAG_DT_SOFTPLUS)
    table, stack, count = _int([[-1] * cap] * R), _int(list(range(R * cap))), _int([R * cap])
    lens = _int([0] * R)
    kc, vc = (torch.full((R * cap, H, page, W), float("nan"), device="cuda") for _ in range(2))
    conv, state = torch.full((R, 3, D), float("nan"), device="cuda"), torch.full((R, D, S), float("nan"), device="cuda")
    outs = [dict(y=torch.zeros(n, D, device="cuda"), a=torch.zeros(n, H, W, device="cuda")) for n in total]
    top = 64
    for step in ([30, 0, 20], [1, 1, 1], [1, 20, 30], [0, 16, 1], [18, 0, 18]):
        p = gdn.gdn_page_plan(table, lens, _int(step), stack, count, page_size=page, max_tokens=top)
        lens, count = p.kv_lens, p.free_count
        rows = [(r, i) for r, i in zip(p.requests.tolist(), p.positions.tolist()) if r >= 0]
        assert len(rows) == sum(step)

        def packed(name):
            t = torch.full((top,) + data[0][name].shape[1:], float("nan"), device="cuda")
            for j, (r, i) in enumerate(rows):
                t[j] = data[r][name][i]
            return t

        where = (kc, vc, table, p.cu_seqlens, lens)
        gdn.gdn_kv_append(packed("k"), packed("v"), *where)
        a = gdn.gdn_paged_attn(packed("q"), *where, max_q=max(step), max_kv=cap * page)
        u, _ = gdn.gdn_causal_conv_fwd(packed("x"), weight, state0=conv, state_final=conv, cu_seqlens=p.cu_seqlens, kv_lens=lens, max_q=max(step), flags=flags["conv"])
        y, _, _ = gdn.gdn_selective_scan_fwd(u, packed("dt"), A, packed("B"), packed("C"), h0=state, h_final=state, cu_seqlens=p.cu_seqlens, kv_lens=lens,
                                             max_q=max(step), flags=flags["scan"])
        held = kc.view(-1, H, page, W)
        for j, (r, i) in enumerate(rows):
            outs[r]["y"][i], outs[r]["a"][i] = y[j], a[j]
            slot = int(p.slots[j])
            assert torch.equal(held[slot // page, :, slot % page], data[r]["k"][i])
        assert not bool(u[len(rows):].any()) and not bool(y[len(rows):].any())
    assert lens.tolist() == total and gdn.gdn_check_device_error() == 0
    for r in range(R):
        d = data[r]
        u, _ = gdn.gdn_causal_conv_fwd(d["x"][None], weight, flags=flags["conv"])
        y, h, _ = gdn.gdn_selective_scan_fwd(u, d["dt"][None], A, d["B"][None], d["C"][None], flags=flags["scan"])
        # the same arithmetic on other tiles and chunks: a few float32 roundings of values of order one
        assert float((outs[r]["y"] - y[0]).abs().max()) <= 2e-4 * float(y.abs().max())
        assert float((state[r] - h[0]).abs().max()) <= 2e-4 * float(h.abs().max())
        x = torch.einsum("qhd,khd->hqk", d["q"].double(), d["k"].double()) * W ** -0.5
        n = total[r]
        x = x.masked_fill(torch.arange(n, device="cuda")[None, :] > torch.arange(n, device="cuda")[:, None], float("-inf"))
        want = torch.einsum("hqk,khd->qhd", torch.softmax(x, -1), d["v"].double())
        assert float((outs[r]["a"].double() - want).norm() / want.norm()) <= 1e-4
