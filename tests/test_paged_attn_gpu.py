"""GPU parity of gdn_paged_attn against the float64 form: lengths and page edges, grouped
heads, ragged chunks, rows without keys, strides, NaN past the lengths, split calls."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn

from paged_reference import Paged, attention, attention_bounds

pytestmark = pytest.mark.gpu


def _run(c, q, scale, **kw):
    kc, vc, table, cu, lens = c.cuda()
    lse = torch.full((c.N, c.Hq), float("nan"), dtype=torch.float32, device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=c.dt, device="cuda")
    kw.setdefault("max_q", max(c.new))
    kw.setdefault("max_kv", max(max(c.length), 1))
    gdn.gdn_paged_attn(q.cuda(), kc, vc, table, cu, lens, scale, out=out, lse=lse, **kw)
    return out.double().cpu(), lse.double().cpu()


def _check(c, q, scale, **kw):
    out, lse = _run(c, q, scale, **kw)
    ref, mag, rlse, size = attention(c, q, scale)
    tol, ltol = attention_bounds(c, ref, mag, rlse, size)
    assert bool(((out - ref).abs() <= tol).all()), float(((out - ref).abs() / tol).max())
    none = torch.isinf(rlse)
    assert bool((lse[none] == -float("inf")).all()) and bool((out[none] == 0).all())
    assert bool(((lse - rlse).abs()[~none] <= ltol.expand_as(rlse)[~none]).all())
    assert gdn.gdn_check_device_error() == 0


SHAPES = [  # new, length
    ([1], [1]),
    ([1, 1, 1], [1, 17, 300]),
    ([1] * 5, [16, 15, 33, 1000, 4097]),
    ([3, 1, 5], [3, 700, 64]),
    ([40, 1, 7], [40, 1500, 130]),
    ([129, 260], [129, 777]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,Hq,Hk,page", [(128, 6, 6, 16), (128, 12, 2, 64), (64, 3, 1, 48), (64, 8, 1, 256)])
@pytest.mark.parametrize("new,length", SHAPES)
def test_matches_float64(dtype, D, Hq, Hk, page, new, length):
    c = Paged(new, length, Hq, Hk, D, page, dtype, seed=len(new) + D)
    _check(c, c.normal(c.N, Hq, D, std=1.5), D ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 5, 16, 17, 40])
def test_group_sizes(dtype, G):
    c = Paged([2, 1, 9], [50, 33, 9], 2 * G, 2, 64, 32, dtype, seed=G)
    _check(c, c.normal(c.N, 2 * G, 64, std=2.0), 0.2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("chunk", [1, 6, 70])
def test_rows_and_sequences_without_keys(dtype, chunk):
    """kv_lens below the new tokens (negative positions), zero lengths and empty sequences."""
    new = [0, chunk, chunk, 0, chunk, 0]
    length = [40, max(chunk - 1, 0), 0, 0, 90, 5]
    c = Paged(new, length, 8, 2, 128, 16, dtype, seed=3)
    _check(c, c.normal(c.N, 8, 128), 128 ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,length", [([1, 1], [200, 61]), ([33, 20], [200, 61])])
def test_strides_of_tokens_and_cache(dtype, new, length):
    """q and out inside wider rows, and a cache stored [page, row, head, channel]."""
    c = Paged(new, length, 12, 4, 128, 32, dtype, seed=5, rows_first=True)
    wide = c.normal(c.N, 20, 128)
    q = wide[:, 8:]
    kc, vc, table, cu, lens = c.cuda()
    assert not kc.is_contiguous()
    out = torch.full((c.N, 14, 128), 7.0, dtype=c.dt, device="cuda")
    gdn.gdn_paged_attn(wide.cuda()[:, 8:], kc, vc, table, cu, lens, 0.1, max_q=max(new), max_kv=max(length),
                       out=out[:, 1:13])
    ref, mag, rlse, size = attention(c, q, 0.1)
    tol, _ = attention_bounds(c, ref, mag, rlse, size)
    assert bool(((out[:, 1:13].double().cpu() - ref).abs() <= tol).all())
    assert bool((out[:, 0] == 7).all()) and bool((out[:, 13] == 7).all())


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_peaked_scores_and_growing_maxima(dtype, D):
    """Scores up to several hundred: the running maximum moves at every step of the pass."""
    c = Paged([1, 50], [900, 640], 4, 2, D, 64, dtype, seed=9)
    q = c.normal(c.N, 4, D)
    for b in range(2):
        n = c.length[b]
        ramp = torch.linspace(0.5, 4.0, n).to(c.dt)
        pages = c.table[b, :-(-n // c.page)].long()
        for i, pg in enumerate(pages.tolist()):
            held = min(c.page, n - i * c.page)
            c.kc[pg, :, :held] = (c.kc[pg, :, :held].float() * ramp[i * c.page:i * c.page + held, None].float()).to(c.dt)
    _check(c, q, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bounds_choose_the_kernel_not_the_result(dtype):
    """Any max_q, max_kv from the exact ones up: the same answer within the bounds."""
    c = Paged([5, 1, 30], [300, 2000, 30], 8, 2, 128, 16, dtype, seed=11)
    q = c.normal(c.N, 8, 128)
    for max_q, max_kv in ((30, 2000), (36, 1 << 20), (1, 1), (1, 100000)):
        _check(c, q, 0.09, max_q=max_q, max_kv=max_kv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_repeats_bitwise_and_any_stream(dtype):
    c = Paged([1] * 7 + [64], [1, 90, 800, 3000, 77, 12, 2049, 400], 16, 2, 128, 64, dtype, seed=13)
    q = c.normal(c.N, 16, 128)
    a, la = _run(c, q, 0.1)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b, lb = _run(c, q, 0.1)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_chunks_agree_with_the_whole_prompt():
    """A prompt in one call, and in chunks over the growing cache."""
    c = Paged([500], [500], 6, 2, 128, 64, "bf16", seed=15)
    q = c.normal(500, 6, 128)
    whole, _ = _run(c, q, 0.1)
    kc, vc, table, _, _ = c.cuda()
    parts, at = [], 0
    for n in (1, 15, 16, 130, 200, 138):
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        lens = torch.tensor([at + n], dtype=torch.int32, device="cuda")
        parts.append(gdn.gdn_paged_attn(q[at:at + n].cuda(), kc, vc, table, cu, lens, 0.1, max_q=n, max_kv=at + n))
        at += n
    ref, mag, rlse, size = attention(c, q, 0.1)
    tol, _ = attention_bounds(c, ref, mag, rlse, size)
    assert bool(((torch.cat(parts).double().cpu() - ref).abs() <= tol).all())
    assert bool(((whole - ref).abs() <= tol).all())


def test_padding_tokens_are_left_alone_and_graphs_replay_with_new_lengths():
    """Rows past cu_seqlens[B] are not written; a captured call reads the arrays anew."""
    c = Paged([2, 3], [40, 200], 8, 2, 128, 16, "bf16", seed=17)
    q = c.normal(9, 8, 128).cuda()
    kc, vc, table, cu, lens = c.cuda()
    out = torch.full((9, 8, 128), 3.0, dtype=c.dt, device="cuda")
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def call():
        gdn.gdn_paged_attn(q, kc, vc, table, cu, lens, 0.1, max_q=3, max_kv=256, out=out, workspace=ws)

    call()
    torch.cuda.synchronize()
    assert bool((out[5:] == 3).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for length in ([40, 200], [17, 5]):
        lens.copy_(torch.tensor(length, dtype=torch.int32))
        out.fill_(3.0)
        graph.replay()
        c.length = length
        ref, mag, rlse, size = attention(c, q[:5].cpu(), 0.1)
        tol, _ = attention_bounds(c, ref, mag, rlse, size)
        assert bool(((out[:5].double().cpu() - ref).abs() <= tol).all())
        assert bool((out[5:] == 3).all())


def test_bad_pages_and_lengths_are_reported():
    """A listed page outside the cache and a length beyond the table: the error word, no stray access."""
    c = Paged([1, 20], [40, 30], 4, 2, 64, 16, "bf16", seed=19)
    q = c.normal(21, 4, 64).cuda()
    kc, vc, table, cu, lens = c.cuda()
    assert gdn.gdn_check_device_error() == 0
    bad = table.clone()
    bad[0, 1] = c.count + 5
    for max_q in (1, 20):
        gdn.gdn_paged_attn(q, kc, vc, bad, cu, lens, 0.1, max_q=max_q, max_kv=64)
        assert gdn.gdn_check_device_error() == gdn.binding.GDN_ERR_INTERNAL
    table[table < 0] = 0
    long = lens.clone()
    long[1] = 100000
    for max_q in (1, 20):
        gdn.gdn_paged_attn(q, kc, vc, table, cu, long, 0.1, max_q=max_q, max_kv=64)
        assert gdn.gdn_check_device_error() == gdn.binding.GDN_ERR_INTERNAL
    assert gdn.gdn_check_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("chunk", [1, 20])
def test_more_sequences_than_a_warp_has_lanes(dtype, chunk):
    new = [chunk if b % 5 else 0 for b in range(70)]
    length = [n + (b * 37) % 400 if n else 0 for b, n in enumerate(new)]
    c = Paged(new, length, 4, 2, 64, 16, dtype, seed=21)
    _check(c, c.normal(c.N, 4, 64), 0.125)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 24])
def test_one_long_sequence_over_every_sm(dtype, new):
    """One item (or two) of 40,000 keys, cut between all CTAs and joined."""
    c = Paged([new], [40000], 6, 1, 64, 64, dtype, seed=23)
    _check(c, c.normal(new, 6, 64), 0.125)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cache_shared_by_all_heads_through_a_zero_stride(dtype):
    """One stored KV head expanded to four (head stride 0)."""
    c = Paged([1, 50], [60, 333], 8, 1, 128, 32, dtype, seed=25)
    q = c.normal(c.N, 8, 128)
    kc, vc, table, cu, lens = c.cuda()
    kc, vc = kc.expand(-1, 4, -1, -1), vc.expand(-1, 4, -1, -1)
    out = gdn.gdn_paged_attn(q.cuda(), kc, vc, table, cu, lens, 0.1, max_q=50, max_kv=333)
    ref, mag, rlse, size = attention(c, q, 0.1)
    tol, _ = attention_bounds(c, ref, mag, rlse, size)
    assert bool(((out.double().cpu() - ref).abs() <= tol).all())


def _device_form(q, kc, vc, cu, lens, table, scale):
    """The same on the GPU in float64, sequence by sequence, for problems too large for the CPU form:
    (out, |v|-weighted out, largest sum |q k| scale)."""
    out, mag = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    size, page, Hk = 0.0, kc.shape[2], kc.shape[1]
    G = q.shape[1] // Hk
    for b in range(len(lens)):
        t0, t1, n = int(cu[b]), int(cu[b + 1]), int(lens[b])
        pages = table[b, :-(-n // page)].long()
        hidden = torch.arange(n, device="cuda")[None, :] > (n - (t1 - t0) + torch.arange(t1 - t0, device="cuda"))[:, None]
        for h in range(Hk):
            k, v = (c[pages, h].reshape(-1, q.shape[2])[:n].double() for c in (kc, vc))
            x = q[t0:t1, h * G:(h + 1) * G].double().transpose(0, 1)
            size = max(size, float((x.abs() @ k.abs().T).max()) * scale)
            p = torch.softmax((x @ k.T * scale).masked_fill(hidden, -float("inf")), -1)
            out[t0:t1, h * G:(h + 1) * G] = (p @ v).transpose(0, 1)
            mag[t0:t1, h * G:(h + 1) * G] = (p @ v.abs()).transpose(0, 1)
    return out.cpu(), mag.cpu(), size


@pytest.mark.parametrize("D,Hq,Hk,new,past", [(128, 48, 8, [700, 1, 513, 40, 1000], [0, 900, 100, 7, 0]),
                                              (64, 24, 24, [1500, 2300, 200], [0, 31, 4000]),
                                              (128, 30, 2, [3000, 130], [250, 1])])
@pytest.mark.parametrize("page", [16, 128])
def test_many_items(D, Hq, Hk, new, past, page):
    """More than two items of 256 rows per SM: a CTA per item; groups that do not divide a tile among them."""
    length = [a + b for a, b in zip(new, past)]
    c = Paged(new, length, Hq, Hk, D, page, "bf16", seed=27)
    q = c.normal(c.N, Hq, D, std=1.5)
    assert c.N * (Hq // Hk) // 256 * Hk >= 304
    kc, vc, table, cu, lens = c.cuda()
    scale = D ** -0.5
    out = gdn.gdn_paged_attn(q.cuda(), kc, vc, table, cu, lens, scale, max_q=max(new), max_kv=max(length)).double().cpu()
    ref, mag, size = _device_form(q.cuda(), kc, vc, c.cu, c.lens, table, scale)
    tol, _ = attention_bounds(c, ref, mag, torch.zeros(1), size)
    assert bool(((out - ref).abs() <= tol).all()), float(((out - ref).abs() / tol).max())
    assert gdn.gdn_check_device_error() == 0
