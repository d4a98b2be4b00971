"""Cases of the operators that feed recurrent layers and the paged cache: the short causal
convolution in front of a recurrent mixer, the selective state space scan, and the plan of a
serving step (page tables, packed offsets and slots from the requests' lengths).

listed() and draw() give cases, prepare() their inputs, run() one pass (plain torch where
``own`` is false, the framework's calls where it is true), exact() the same in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # One decoding step of a full batch: q, k and v of 48 heads, states in a pool.
        dict(name="conv_step", op="conv", train=False, seqs=32, new=1, past=True, channels=18432, taps=4, silu=True,
             bias=False, pad=0, dtype="bf16"),
        # A prefill step of six packed ragged sequences, some with a past, padded for a captured graph.
        dict(name="conv_prompts", op="conv", train=False, seqs=6, new=4096, past=True, channels=6144, taps=4, silu=True,
             bias=True, pad=100, dtype="bf16"),
        # Training step at batch 8, 4096 tokens: q, k and v of 6 heads in one call, forward and backward.
        dict(name="conv_train", op="conv", train=True, seqs=8, new=4096, past=False, channels=2304, taps=4, silu=True,
             bias=False, pad=0, dtype="bf16"),
        # Single precision, odd sizes, no activation, carried states: the checking configuration.
        dict(name="conv_train_f32", op="conv", train=True, seqs=3, new=1021, past=True, channels=1001, taps=3,
             silu=False, bias=True, pad=0, dtype="f32"),
        # One sequence decoding alone: latency.
        dict(name="scan_one", op="scan", train=False, seqs=1, new=1, past=True, channels=768, states=16, groups=1,
             gate=True, pad=0, dtype="bf16"),
        # One decoding step of a full batch, states in a pool: bandwidth.
        dict(name="scan_step", op="scan", train=False, seqs=32, new=1, past=True, channels=6144, states=16, groups=1,
             gate=True, pad=0, dtype="bf16"),
        # One long prompt: few channels, many tokens.
        dict(name="scan_long", op="scan", train=False, seqs=1, new=32768, past=False, channels=2048, states=16, groups=1,
             gate=True, pad=0, dtype="bf16"),
        # A prefill step of six packed ragged sequences, some with a past, padded for a captured graph.
        dict(name="scan_prompts", op="scan", train=False, seqs=6, new=4096, past=True, channels=6144, states=16, groups=1,
             gate=True, pad=100, dtype="bf16"),
        # Training step at batch 8, 4096 tokens, forward and backward.
        dict(name="scan_train", op="scan", train=True, seqs=8, new=4096, past=False, channels=768, states=16, groups=1,
             gate=True, pad=0, dtype="bf16"),
        # Single precision, odd sizes, wide states in groups, no gate, carried states.
        dict(name="scan_train_f32", op="scan", train=True, seqs=2, new=517, past=True, channels=1002, states=64, groups=2,
             gate=False, pad=0, dtype="f32"),
        # One decoding step of a full batch: a token each, few new pages.
        dict(name="plan_step", op="plan", requests=256, new=1, length=4096, page=64, max_tokens=256, spare=1.0),
        # Prompts, drafts, rejected drafts and finished requests in one step, pages running out.
        dict(name="plan_mixed", op="plan", requests=1024, new=4096, length=32768, page=16, max_tokens=131072, spare=0.9),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv", "scan", "scan", "plan"])
    if op == "plan":
        new = rng.choice([1, rng.randint(2, 16), _log_int(rng, 17, 4096)])
        requests = _log_int(rng, 1, 1024)
        top = requests if new == 1 else min(131072, max(16, requests * new // 4))
        return dict(op=op, requests=requests, new=new, length=_log_int(rng, 64, 32768), page=rng.choice([16, 48, 64, 256]),
                    max_tokens=top, spare=rng.choice([1.0, 1.0, 0.9]))
    train = rng.random() < 0.4
    dtype = rng.choice(["bf16", "bf16", "f32"])
    shape = rng.choice(["step", "draft", "prompt", "prompt"])
    new = _log_int(rng, 17, 4096)
    if not train and shape != "prompt":
        new = 1 if shape == "step" else rng.randint(2, 16)
    elif not train and rng.random() < 0.25:
        new = _log_int(rng, 4097, 32768)
    c = dict(op=op, train=train, seqs=_log_int(rng, 1, 64), new=new, past=rng.random() < 0.6)
    channels = _log_int(rng, 64, 8192)
    if rng.random() < 0.7:
        channels = max(64, channels // 64 * 64)
    if op == "conv":
        c.update(channels=channels, taps=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.7, bias=rng.random() < 0.5)
        most = 32768 * 2304 * 2 // BYTES[dtype] // channels
    else:
        groups = rng.choice([1, 1, 1, 2, 4])
        channels = max(groups, channels // groups * groups)
        c.update(channels=channels, states=rng.choice([8, 16, 16, 16, 32, 64]), groups=groups, gate=rng.random() < 0.7)
        most = (32768 * 768 * 16 if train else 32768 * 2048 * 16) // (channels * c["states"])
    c["new"] = max(1, min(c["new"], most))
    c["seqs"] = max(1, min(c["seqs"], most // c["new"]))
    c.update(pad=0 if train else rng.choice([0, rng.randint(1, 64)]), dtype=dtype)
    return c


def _lengths(case):
    """New tokens of each sequence: the last has the case's full size, in packed prompts the others
    from a sixteenth of it up, in a fixed mixed order."""
    n, top = case["seqs"], case["new"]
    if case["train"] or top <= 16:
        return [top] * n
    share = [1.0 if b == n - 1 else 1 / 16 + 15 / 16 * ((7 * b + 3) % n + 1) / n for b in range(n)]
    return [max(1, int(top * s)) for s in share]


def work(case):
    if case["op"] == "plan":
        tokens = min(case["max_tokens"], case["requests"] * case["new"])
        pages = tokens // case["page"] + case["requests"]
        return {"bytes": case["requests"] * 16 + pages * 8 + case["max_tokens"] * 16, "flops": 8 * tokens}
    e, tokens, d = BYTES[case["dtype"]], sum(_lengths(case)), case["channels"]
    if case["op"] == "conv":
        held = case["seqs"] * (case["taps"] - 1) * d * e * (1 + case["past"])
        if not case["train"]:
            return {"bytes": 2 * tokens * d * e + held, "flops": tokens * d * (2 * case["taps"] + 5)}
        return {"bytes": 5 * tokens * d * e + 2 * held, "flops": tokens * d * (8 * case["taps"] + 15)}
    held = case["seqs"] * d * case["states"] * 4 * (1 + case["past"])
    ins = tokens * e * (d * (2 + case["gate"]) + 2 * case["groups"] * case["states"])
    inner = tokens * d * case["states"]
    if not case["train"]:
        return {"bytes": ins + tokens * d * e + held, "flops": 8 * inner + 12 * tokens * d}
    return {"bytes": 3 * ins + 2 * tokens * d * e + 2 * held, "flops": 32 * inner + 40 * tokens * d}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case=dict(case))

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=gen, device="cuda")

    if case["op"] == "plan":
        n, page = case["requests"], case["page"]
        cap = -(-(case["length"] + case["new"]) // page)
        lens = (case["length"] * uniform(n) ** 2).long()
        used = (lens + page - 1) // page
        kind = uniform(n)
        new = torch.ones(n, dtype=torch.long, device="cuda")
        if case["new"] > 1:
            # some idle, some finished, some giving back drafts, decoding ones, and prompts
            size = (case["new"] * uniform(n) ** 3).long() + 1
            back = -torch.minimum(whole(1, 8, n), lens)
            new = torch.where(kind < 0.1, 0 * new, torch.where(kind < 0.15, -lens, torch.where(
                kind < 0.25, back, torch.where(kind < 0.6, new, size))))
        need = ((lens + new.clamp(min=0) + page - 1) // page - used).sum()
        held = int(used.sum())
        free = int(need * case["spare"]) + (5 if case["spare"] >= 1 else 0)
        pages = n * cap + 6
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        col = torch.arange(cap, device="cuda")
        at = (used.cumsum(0) - used)[:, None] + col[None, :]
        mine = col[None, :] < used[:, None]
        s["page_table"] = torch.where(mine, order[at.clamp(max=pages - 1)], torch.full_like(at, -1, dtype=torch.int32))
        s["free_pages"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        s["free_pages"][:free] = order[held:held + free]
        s["free_count"] = torch.tensor([free], dtype=torch.int32, device="cuda")
        s["kv_lens"], s["new_tokens"] = lens.to(torch.int32), new.to(torch.int32)
        return s

    dt = DTYPES[case["dtype"]]

    def normal(*shape, mean=0.0, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std).add_(mean)

    n, d, new = case["seqs"], case["channels"], _lengths(case)
    rows = sum(new) + case["pad"]
    lead = (n, case["new"]) if case["train"] else (rows,)
    if not case["train"]:
        s["cu_seqlens"] = torch.tensor([sum(new[:b]) for b in range(n + 1)], dtype=torch.int32, device="cuda")
        # every third sequence starts here; the others have a past, and states in a pool
        past = [0 if not case["past"] or b % 3 == 1 else 17 + b for b in range(n)]
        s["kv_lens"] = torch.tensor([a + b for a, b in zip(new, past)], dtype=torch.int32, device="cuda")
        s["slots"] = torch.randperm(n + 3, generator=gen, device="cuda")[:n].to(torch.int32)
        s["max_q"] = max(new)
    pool = n if case["train"] else n + 3
    if case["op"] == "conv":
        k = case["taps"]
        s["x"] = normal(*lead, d).to(dt)
        s["weight"] = normal(d, k, std=k ** -0.5).to(dt)
        s["bias"] = normal(d, std=0.2).to(dt) if case["bias"] else None
        s["state0"] = normal(pool, k - 1, d).to(dt) if case["past"] or not case["train"] else None
        if case["train"]:
            s["dy"] = normal(*lead, d).to(dt)
            s["dstate"] = normal(n, k - 1, d, std=0.5).to(dt) if case["past"] else None
        else:
            s["state_out"] = torch.zeros_like(s["state0"])  # another pool, so that a step can be taken back
        return s
    m, g = case["states"], case["groups"]
    s["u"] = normal(*lead, d).to(dt)
    s["dt"] = normal(*lead, d, std=0.5).to(dt)
    # B and C are views of one projection
    bc = normal(*lead, 2 * g * m).to(dt)
    s["B"], s["C"] = (t.unflatten(-1, (g, m)) for t in bc.split(g * m, -1))
    s["A"] = -torch.arange(1, m + 1, device="cuda") * normal(d, m, std=0.1).exp_()
    s["D"] = normal(d, mean=1.0, std=0.1)
    # steps of 0.001 to 0.1 at dt = 0
    s["dt_bias"] = torch.expm1(torch.exp(math.log(1e-3) + math.log(100.0) * uniform(d))).log()
    s["z"] = normal(*lead, d).to(dt) if case["gate"] else None
    s["h0"] = normal(pool, d, m) if case["past"] or not case["train"] else None
    if case["train"]:
        s["dy"] = normal(*lead, d).to(dt)
        s["dh"] = normal(n, d, m, std=0.1) if case["past"] else None
    else:
        s["h_out"] = torch.zeros_like(s["h0"])
    return s


# ---------------------------------------------------------------- plain forms (32 bits)
def _places(s, rows):
    """(sequence, index in it) of every row, its length, whether a sequence has a state; rows behind the last
    sequence belong to none (sequence -1)."""
    case = s["case"]
    row = torch.arange(rows, device="cuda")
    if case["train"]:
        t = case["new"]
        return row // t, row % t, torch.full((case["seqs"],), t, device="cuda"), torch.ones(
            case["seqs"], dtype=torch.bool, device="cuda")
    cu = s["cu_seqlens"].long()
    b = torch.searchsorted(cu, row, right=True) - 1
    real = row < cu[-1]
    new = cu[1:] - cu[:-1]
    return torch.where(real, b, -1), torch.where(real, row - cu[b.clamp(max=case["seqs"] - 1)], 0), new, s["kv_lens"] > new


def _conv_plain(s):
    case = s["case"]
    k, dt = case["taps"], s["x"].dtype
    x = s["x"].flatten(0, -2).float()
    rows, d = x.shape
    b, i, new, old = _places(s, rows)
    n = case["seqs"]
    first = new.cumsum(0) - new
    if s["state0"] is None:
        held = torch.zeros(n, k - 1, d, device="cuda")
    else:
        held = s["state0"].float() if case["train"] else s["state0"].float()[s["slots"].long()]
        held = torch.where(old[:, None, None], held, torch.zeros_like(held))
    # every sequence with its held inputs in front: [row of the sequence, its inputs]
    every = torch.cat((held.flatten(0, 1), x))
    back = torch.arange(k, device="cuda") - (k - 1)
    at = i[:, None] + back[None, :]
    here = torch.where(at >= 0, (n * (k - 1) + torch.arange(rows, device="cuda"))[:, None] + back[None, :],
                       b.clamp(min=0)[:, None] * (k - 1) + at + k - 1)
    taps = every[here.clamp(min=0)]  # [rows, k, d]
    w = s["weight"].float()
    pre = (taps * w.T[None]).sum(1)
    if s["bias"] is not None:
        pre = pre + s["bias"].float()
    sig = 1.0 / (1.0 + torch.exp(-pre))
    real = (b >= 0)[:, None]
    y = torch.where(real, pre * sig if case["silu"] else pre, torch.zeros_like(pre))
    out = {"y": y.view(s["x"].shape).to(dt)}
    tail = new[:, None] + back[None, :-1]
    src = torch.where(tail >= 0, n * (k - 1) + first[:, None] + tail,
                      torch.arange(n, device="cuda")[:, None] * (k - 1) + tail + k - 1)
    last = every[src.clamp(min=0)].to(dt)
    if not case["train"]:
        s["state_out"][s["slots"].long()] = last
        out["state"] = s["state_out"]
        return out
    out["state"] = last
    dpre = s["dy"].flatten(0, -2).float()
    if case["silu"]:
        dpre = dpre * sig * (1.0 + pre * (1.0 - sig))
    out["dweight"] = (dpre[:, None, :] * taps).sum(0).T.to(dt)
    if s["bias"] is not None:
        out["dbias"] = dpre.sum(0).to(dt)
    # sequences are equally long in training: the gradient of an input is a sum over the taps that read it
    full = torch.zeros(n, case["new"] + k - 1, k, d, device="cuda")
    full[:, :case["new"]] = dpre.view(n, case["new"], 1, d) * w.T
    col = torch.arange(case["new"] + k - 1, device="cuda")[:, None] - torch.arange(k, device="cuda")[None, :]
    ext = torch.where((col >= 0)[None, :, :, None], full[:, col.clamp(min=0), torch.arange(k, device="cuda")],
                      torch.zeros((), device="cuda")).sum(2)
    if s["dstate"] is not None:
        ext[:, case["new"]:] += s["dstate"].float()
    out["dx"] = ext[:, k - 1:].reshape(s["x"].shape).to(dt)
    if s["state0"] is not None:
        out["dstate0"] = ext[:, :k - 1].to(dt)
    return out


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first dimension, h_{-1} = 0: neighbours are joined, the joined ones
    scanned, and the ones between filled in."""
    t = a.shape[0]
    if t == 1:
        return b
    even = t // 2 * 2
    a0, b0, a1, b1 = a[0:even:2], b[0:even:2], a[1:even:2], b[1:even:2]
    odd = _scan(a0 * a1, torch.addcmul(b1, a1, b0))
    h = torch.empty_like(b)
    h[1:even:2] = odd
    h[0] = b[0]
    rest = a[2::2]
    h[2::2] = torch.addcmul(b[2::2], rest, odd[:rest.shape[0]])
    return h


def _scan_plain(s):
    case, dt = s["case"], s["u"].dtype
    m, g, d = case["states"], case["groups"], case["channels"]
    u, raw = s["u"].flatten(0, -2).float(), s["dt"].flatten(0, -2).float() + s["dt_bias"]
    rows = u.shape[0]
    b, i, new, old = _places(s, rows)
    real, first = b >= 0, i == 0
    delta = raw.clamp(min=0) + torch.log1p(torch.exp(-raw.abs()))
    delta = torch.where(real[:, None], delta, torch.zeros_like(delta))

    def spread(t):  # [rows, g, m] -> [rows, d, m]
        return t.reshape(rows, g, m).float().repeat_interleave(d // g, 1)

    bm, cm = spread(s["B"]), spread(s["C"])
    a = torch.exp(delta[:, :, None] * s["A"])
    x = bm * (delta * u)[:, :, None]
    if s["h0"] is not None:
        held = s["h0"] if case["train"] else s["h0"][s["slots"].long()]
        held = torch.where(old[:, None, None], held, torch.zeros_like(held))
        start = new.cumsum(0) - new
        x[start] += a[start] * held
    cut = torch.where((first & real)[:, None, None], torch.zeros((), device="cuda"), a)
    h = _scan(cut, x)
    c = (h * cm).sum(-1)
    y = c + u * s["D"]
    if case["gate"]:
        z = s["z"].flatten(0, -2).float()
        sig = 1.0 / (1.0 + torch.exp(-z))
        act = z * sig
    out = {"y": torch.where(real[:, None], y * act if case["gate"] else y, torch.zeros_like(y)).view(s["u"].shape).to(dt)}
    end = new.cumsum(0) - 1
    last = h[end]
    if not case["train"]:
        s["h_out"][s["slots"].long()] = last
        out["h"] = s["h_out"]
        return out
    out["h"] = last
    dy = s["dy"].flatten(0, -2).float()
    if case["gate"]:
        out["dz"] = (dy * y * sig * (1.0 + z * (1.0 - sig))).view(s["u"].shape).to(dt)
        dy = dy * act
    out["dD"] = (dy * u).sum(0)
    gx = cm * dy[:, :, None]
    if s["dh"] is not None:
        gx[end] += s["dh"]
    after = torch.zeros_like(cut)
    after[:-1] = cut[1:]
    gh = _scan(after.flip(0), gx.flip(0)).flip(0)
    out["dC"] = (h * dy[:, :, None]).view(rows, g, d // g, m).sum(2).view(s["C"].shape).to(dt)
    out["dB"] = (gh * (delta * u)[:, :, None]).view(rows, g, d // g, m).sum(2).view(s["B"].shape).to(dt)
    dx = (gh * bm).sum(-1)
    del after, gx, cm
    before = torch.cat((torch.zeros_like(h[:1]), h[:-1]))
    before[new.cumsum(0) - new] = 0 if s["h0"] is None else held
    ga = gh * a * before
    out["dA"] = (ga * delta[:, :, None]).sum(0)
    ddelta = (ga * s["A"]).sum(-1) + dx * u
    draw_ = ddelta / (1.0 + torch.exp(-raw))
    out["du"] = (dx * delta + dy * s["D"]).view(s["u"].shape).to(dt)
    out["ddt"] = draw_.view(s["u"].shape).to(dt)
    out["ddt_bias"] = draw_.sum(0)
    if s["h0"] is not None:
        begin = new.cumsum(0) - new
        out["dh0"] = gh[begin] * a[begin]
    return out


def _plan_plain(s):
    case = s["case"]
    n, page, top = case["requests"], case["page"], case["max_tokens"]
    table, lens, new = s["page_table"], s["kv_lens"].long(), s["new_tokens"].long()
    cap = table.shape[1]
    count = s["free_count"].long()
    used = (lens + page - 1) // page
    left = torch.where(new < 0, (lens + new).clamp(min=0), lens)
    keep = (left + page - 1) // page
    back = used - keep
    col = torch.arange(cap, device="cuda")[None, :]
    gone = (col >= keep[:, None]) & (col < used[:, None])
    order = gone.flatten().cumsum(0) - 1
    at = torch.where(gone.flatten(), count + order, s["free_pages"].shape[0])
    ext = torch.cat((s["free_pages"], s["free_pages"].new_zeros(1)))
    ext[at] = torch.where(gone.flatten(), table.flatten(), ext[-1])
    s["free_pages"].copy_(ext[:-1])
    have = count + back.sum()
    ask = new.clamp(min=0)
    fits = lens + ask <= cap * page
    ask = torch.where(fits, ask, 0)
    need = (lens + ask + page - 1) // page - used
    need = torch.where(ask > 0, need, 0)
    got = ((need == 0) | (need.cumsum(0) <= have)) & (ask.cumsum(0) <= top)
    ask, need = torch.where(got, ask, 0), torch.where(got, need, 0)
    cum = need.cumsum(0) - need
    fresh = (col >= used[:, None]) & (col < (used + need)[:, None])
    which = (have - 1 - (cum[:, None] + col - used[:, None])).clamp(min=0, max=s["free_pages"].shape[0] - 1)
    table.copy_(torch.where(fresh, s["free_pages"][which], table))
    cu = torch.cat((ask.new_zeros(1), ask.cumsum(0)))
    tok = torch.arange(top, device="cuda")
    r = torch.searchsorted(cu, tok, right=True) - 1
    real = tok < cu[-1]
    r = torch.where(real, r, 0)
    pos = lens[r] + tok - cu[r]
    slot = table[r, torch.where(real, pos // page, 0)].long() * page + pos % page
    none = torch.full_like(tok, -1)
    return {"cu_seqlens": cu.to(torch.int32), "kv_lens": (left + ask).to(torch.int32),
            "free_count": (have - need.sum()).to(torch.int32), "requests": torch.where(real, r, none).to(torch.int32),
            "positions": torch.where(real, pos, none).to(torch.int32), "slots": torch.where(real, slot, none),
            "page_table": table, "free_pages": s["free_pages"]}


# ---------------------------------------------------------------- the framework's calls
def _conv_own(s):
    import gated_deltanet_gdn_gb300 as gdn

    case = s["case"]
    flags = gdn.GDN_FLAG_CONV_SILU if case["silu"] else 0
    if not case["train"]:
        y, state = gdn.gdn_causal_conv_fwd(s["x"], s["weight"], s["bias"], state0=s["state0"], state_final=s["state_out"],
                                           slots=s["slots"], cu_seqlens=s["cu_seqlens"], kv_lens=s["kv_lens"],
                                           max_q=s["max_q"], flags=flags)
        return {"y": y, "state": state}
    y, state = gdn.gdn_causal_conv_fwd(s["x"], s["weight"], s["bias"], state0=s["state0"], flags=flags)
    grads = gdn.gdn_causal_conv_bwd(s["x"], s["weight"], s["bias"], s["dy"], state0=s["state0"], dstate=s["dstate"],
                                    flags=flags)
    return {"y": y, "state": state, **{k: v for k, v in grads.items() if v is not None}}


def _scan_own(s):
    import gated_deltanet_gdn_gb300 as gdn

    case, flags = s["case"], gdn.GDN_FLAG_DT_SOFTPLUS
    args = (s["u"], s["dt"], s["A"], s["B"], s["C"])
    parts = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    if not case["train"]:
        y, h, _ = gdn.gdn_selective_scan_fwd(*args, **parts, h0=s["h0"], h_final=s["h_out"], slots=s["slots"],
                                             cu_seqlens=s["cu_seqlens"], kv_lens=s["kv_lens"], max_q=s["max_q"], flags=flags)
        return {"y": y, "h": h}
    y, h, kept = gdn.gdn_selective_scan_fwd(*args, **parts, h0=s["h0"], flags=flags, save=True)
    grads = gdn.gdn_selective_scan_bwd(*args, s["dy"], kept, **parts, dh_final=s["dh"], need_dh0=s["h0"] is not None,
                                       flags=flags)
    return {"y": y, "h": h, **{k: v for k, v in grads.items() if v is not None}}


def _plan_own(s):
    import gated_deltanet_gdn_gb300 as gdn

    p = gdn.gdn_page_plan(s["page_table"], s["kv_lens"], s["new_tokens"], s["free_pages"], s["free_count"],
                          page_size=s["case"]["page"], max_tokens=s["case"]["max_tokens"])
    return {"cu_seqlens": p.cu_seqlens, "kv_lens": p.kv_lens, "free_count": p.free_count, "requests": p.requests,
            "positions": p.positions, "slots": p.slots, "page_table": s["page_table"], "free_pages": s["free_pages"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"conv": _conv_own, "scan": _scan_own, "plan": _plan_own}[op](state)
    return {"conv": _conv_plain, "scan": _scan_plain, "plan": _plan_plain}[op](state)


# ---------------------------------------------------------------- 64 bits, from the definitions
def _exact_conv(s):
    """Sequence by sequence: shifted products of the padded inputs, gradients by reverse differentiation."""
    case = s["case"]
    k, n, new = case["taps"], case["seqs"], _lengths(case)
    leaf = {"x": s["x"].double().requires_grad_(), "weight": s["weight"].double().requires_grad_()}
    if s["bias"] is not None:
        leaf["bias"] = s["bias"].double().requires_grad_()
    if s["state0"] is not None and case["train"]:
        leaf["state0"] = s["state0"].double().requires_grad_()
    x = leaf["x"].flatten(0, -2)
    ys, states, at = [], [], 0
    for b in range(n):
        held = torch.zeros(k - 1, case["channels"], dtype=torch.float64, device="cuda")
        if case["train"] and s["state0"] is not None:
            held = leaf["state0"][b]
        elif not case["train"] and int(s["kv_lens"][b]) > new[b]:
            held = s["state0"][int(s["slots"][b])].double()
        seq = torch.cat((held, x[at:at + new[b]]))
        pre = sum(seq[j:j + new[b]] * leaf["weight"][:, j] for j in range(k))
        pre = pre + leaf["bias"] if "bias" in leaf else pre
        ys.append(pre * torch.sigmoid(pre) if case["silu"] else pre)
        states.append(seq[new[b]:])
        at += new[b]
    ys.append(torch.zeros(case["pad"], case["channels"], dtype=torch.float64, device="cuda"))
    y = torch.cat(ys).view(s["x"].shape)
    if not case["train"]:
        state = s["state_out"].double()
        state[s["slots"].long()] = torch.stack(states).detach()
        return {"y": y.detach(), "state": state}
    state = torch.stack(states)
    loss = (y * s["dy"].double()).sum()
    if s["dstate"] is not None:
        loss = loss + (state * s["dstate"].double()).sum()
    grads = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))
    out = {"y": y.detach(), "state": state.detach(), "dweight": grads["weight"]}
    if "bias" in grads:
        out["dbias"] = grads["bias"]
    out["dx"] = grads["x"]
    if "state0" in grads:
        out["dstate0"] = grads["state0"]
    return out


def _steps(a, x):
    """h_t = a_t h_{t-1} + x_t along the first dimension by doubling: after step j every element holds the
    sum of its last 2^j terms and the product of their factors."""
    a, x, j = a.clone(), x.clone(), 1
    while j < x.shape[0]:
        x[j:] = x[j:] + a[j:] * x[:-j]
        a[j:] = a[j:] * a[:-j]
        j *= 2
    return x


def _exact_scan(s):
    """Sequence by sequence and a block of channels at a time; the gradients as sums over the states' adjoints
    p_t = C_t dy_t + a_{t+1} p_{t+1}."""
    case = s["case"]
    m, g, d, n, train = case["states"], case["groups"], case["channels"], case["seqs"], case["train"]
    new = _lengths(case)
    flat = {k: s[k].flatten(0, -2) for k in ("u", "dt")}
    gate = s["z"].flatten(0, -2) if case["gate"] else None
    bm, cm = (s[k].reshape(-1, g, m) for k in ("B", "C"))
    dyr = s["dy"].flatten(0, -2) if train else None
    like = dict(dtype=torch.float64, device="cuda")
    rows = flat["u"].shape[0]
    y = torch.zeros(rows, d, **like)
    h_last = torch.zeros(n, d, m, **like)
    out = {k: torch.zeros(rows, d, **like) for k in ("dz", "du", "ddt")} if train else {}
    if train:
        out.update(dD=torch.zeros(d, **like), ddt_bias=torch.zeros(d, **like), dA=torch.zeros(d, m, **like),
                   dB=torch.zeros(rows, g, m, **like), dC=torch.zeros(rows, g, m, **like), dh0=torch.zeros(n, d, m, **like))
    at = 0
    for b in range(n):
        rs = slice(at, at + new[b])
        wide = max(1, 2 ** 26 // (new[b] * m))
        for q in range(g):
            for lo in range(q * d // g, (q + 1) * d // g, wide):
                cs = slice(lo, min(lo + wide, (q + 1) * d // g))
                u, raw = flat["u"][rs, cs].double(), flat["dt"][rs, cs].double() + s["dt_bias"][cs].double()
                step = torch.nn.functional.softplus(raw, threshold=700.0)
                bq, cq = bm[rs, q].double()[:, None, :], cm[rs, q].double()[:, None, :]
                amat = s["A"][cs].double()
                a = torch.exp(step[:, :, None] * amat)
                x = (step * u)[:, :, None] * bq
                h0 = None
                if train and s["h0"] is not None:
                    h0 = s["h0"][b, cs].double()
                elif not train and int(s["kv_lens"][b]) > new[b]:
                    h0 = s["h0"][int(s["slots"][b]), cs].double()
                if h0 is not None:
                    x[0] = x[0] + a[0] * h0
                h = _steps(a, x)
                h_last[b, cs] = h[-1]
                yc = torch.einsum("tdm,tm->td", h, cq[:, 0]) + u * s["D"][cs].double()
                z = gate[rs, cs].double() if case["gate"] else None
                y[rs, cs] = yc * z * torch.sigmoid(z) if case["gate"] else yc
                if not train:
                    continue
                dy = dyr[rs, cs].double()
                if case["gate"]:
                    sg = torch.sigmoid(z)
                    out["dz"][rs, cs] = dy * yc * (sg + z * sg * (1 - sg))
                    dy = dy * z * sg
                p = dy[:, :, None] * cq
                if s["dh"] is not None:
                    p[-1] = p[-1] + s["dh"][b, cs].double()
                shift = torch.cat((a[1:], torch.zeros_like(a[:1])))
                p = _steps(shift.flip(0), p.flip(0)).flip(0)
                prev = torch.cat((torch.zeros_like(h[:1]) if h0 is None else h0[None], h[:-1]))
                dlog = p * a * prev
                out["dh0"][b, cs] = p[0] * a[0]
                out["dA"][cs] += torch.einsum("tdm,td->dm", dlog, step)
                out["dC"][rs, q] += torch.einsum("tdm,td->tm", h, dy)
                out["dB"][rs, q] += torch.einsum("tdm,td->tm", p, step * u)
                through = torch.einsum("tdm,tm->td", p, bq[:, 0])
                out["dD"][cs] += (dy * u).sum(0)
                out["du"][rs, cs] = through * step + dy * s["D"][cs].double()
                dstep = (torch.einsum("tdm,dm->td", dlog, amat) + through * u) * torch.sigmoid(raw)
                out["ddt"][rs, cs] = dstep
                out["ddt_bias"][cs] += dstep.sum(0)
        at += new[b]
    first = {"y": y.view(s["u"].shape)}
    if not train:
        state = s["h_out"].double()
        state[s["slots"].long()] = h_last
        return {**first, "h": state}
    first["h"] = h_last
    if case["gate"]:
        first["dz"] = out["dz"].view(s["u"].shape)
    first.update(dD=out["dD"], dC=out["dC"].view(s["C"].shape), dB=out["dB"].view(s["B"].shape), dA=out["dA"],
                 du=out["du"].view(s["u"].shape), ddt=out["ddt"].view(s["u"].shape), ddt_bias=out["ddt_bias"])
    if s["h0"] is not None:
        first["dh0"] = out["dh0"]
    return first


def _exact_plan(s):
    """Request by request, with a list for a stack."""
    case = s["case"]
    n, page, top = case["requests"], case["page"], case["max_tokens"]
    table, lens, new = s["page_table"].cpu().tolist(), s["kv_lens"].tolist(), s["new_tokens"].tolist()
    slots = s["free_pages"].tolist()
    stack = slots[:int(s["free_count"])]
    kept = list(lens)
    for b in range(n):
        if new[b] < 0:
            kept[b] = max(0, lens[b] + new[b])
            stack += table[b][-(-kept[b] // page):-(-lens[b] // page)]
    slots[:len(stack)] = stack
    have, asked, tokens = len(stack), 0, 0
    cu, where = [0], []
    for b in range(n):
        ask = new[b] if 0 < new[b] <= len(table[b]) * page - lens[b] else 0
        pages = -(-(lens[b] + ask) // page) + (lens[b] // -page) if ask else 0
        asked, tokens = asked + pages, tokens + ask
        if (pages and asked > have) or tokens > top:
            ask = pages = 0
        for j in range(pages):
            table[b][-(-lens[b] // page) + j] = stack.pop()
        where += [(b, lens[b] + i, table[b][(lens[b] + i) // page] * page + (lens[b] + i) % page) for i in range(ask)]
        kept[b] += ask
        cu.append(cu[-1] + ask)
    where += [(-1, -1, -1)] * (top - len(where))
    r, pos, slot = zip(*where)

    def put(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device="cuda")

    return {"cu_seqlens": put(cu), "kv_lens": put(kept), "free_count": put([len(stack)]), "requests": put(r),
            "positions": put(pos), "slots": put(slot, torch.int64), "page_table": put(table), "free_pages": put(slots)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "plan": _exact_plan}[case["op"]](s)
