"""Cases of the operators that a hybrid stack runs beside the gated delta rule: appending to
a paged key/value cache with the position rotation, attention of new tokens over that cache,
and the norms around a block with its gate and residual scale (forward, and with backward).

listed() and draw() give cases, prepare() their inputs, run() one pass (plain torch where
``own`` is false, the framework's calls where it is true), exact() the same in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-6


def listed():
    return [
        # One decoding step of a full batch: the append in front of every attention layer.
        dict(name="append_step", op="append", seqs=32, chunk=1, past=4096, q_heads=48, kv_heads=8, width=128,
             page=64, rot=128, pairs=False, dtype="bf16"),
        # A prefill step of four packed sequences (ragged, with a past), rows taken from one fused projection.
        dict(name="append_prefill", op="append", seqs=4, chunk=8192, past=1500, q_heads=48, kv_heads=8, width=128,
             page=64, rot=64, pairs=True, dtype="bf16"),
        # One sequence decoding alone: latency.
        dict(name="attn_one", op="attn", seqs=1, chunk=1, past=2047, q_heads=6, kv_heads=6, width=128, page=64,
             dtype="bf16"),
        # One decoding step of a full batch with long ragged contexts: bandwidth.
        dict(name="attn_step", op="attn", seqs=32, chunk=1, past=32767, q_heads=48, kv_heads=8, width=128, page=64,
             dtype="bf16"),
        # Eight draft tokens per sequence checked at once, pages of 48 tokens.
        dict(name="attn_draft", op="attn", seqs=16, chunk=8, past=16000, q_heads=16, kv_heads=2, width=128, page=48,
             dtype="bf16"),
        # A late chunk of one long prompt: compute.
        dict(name="attn_chunk", op="attn", seqs=1, chunk=2048, past=63488, q_heads=16, kv_heads=4, width=128,
             page=128, dtype="bf16"),
        # Whole packed prompts of different lengths, nothing cached before.
        dict(name="attn_prompts", op="attn", seqs=6, chunk=4096, past=0, q_heads=48, kv_heads=8, width=128, page=16,
             dtype="bf16"),
        # Single precision, narrow heads in groups of three, short chunks: the checking configuration.
        dict(name="attn_f32", op="attn", seqs=3, chunk=200, past=1301, q_heads=6, kv_heads=2, width=64, page=16,
             dtype="f32"),
        # The gated norm of every head's output in one decoding step.
        dict(name="norm_step", op="norm", train=False, rows=32, groups=48, width=128, post=True, gate=True,
             residual=False, scale=False, pre=False, dtype="bf16"),
        # The same in a training step at batch 8, 4096 tokens, 6 heads.
        dict(name="norm_heads", op="norm", train=True, rows=32768, groups=6, width=128, post=True, gate=True,
             residual=False, scale=False, pre=False, dtype="bf16"),
        # Between two blocks of a 48-head model in training: norm after, gate, scaled residual, norm before.
        dict(name="norm_block", op="norm", train=True, rows=8192, groups=1, width=6144, post=True, gate=True,
             residual=True, scale=True, pre=True, dtype="bf16"),
        # Single precision, an odd width, no gate: residual scale and the next block's norm only.
        dict(name="norm_f32", op="norm", train=True, rows=1021, groups=1, width=1001, post=False, gate=False,
             residual=True, scale=True, pre=True, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "attn", "attn", "norm"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if kind == "norm":
        train, heads = rng.random() < 0.6, rng.random() < 0.4
        if heads:
            rows, groups, width = _log_int(rng, 1, 32768), rng.choice([1, 2, 6, 16, 48]), rng.choice([64, 128])
            rows = max(1, min(rows, 32768 * 6 * 128 // (groups * width)))
            return dict(op="norm", train=train, rows=rows, groups=groups, width=width, post=True, gate=True,
                        residual=False, scale=False, pre=False, dtype=dtype)
        width = _log_int(rng, 96, 8192)
        if rng.random() < 0.7:
            width = max(64, width // 64 * 64)
        rows = min(_log_int(rng, 1, 16384), 8192 * 6144 // (width * BYTES[dtype] // 2))
        post, residual = rng.random() < 0.6, rng.random() < 0.8
        return dict(op="norm", train=train, rows=max(1, rows), groups=1, width=width, post=post,
                    gate=rng.random() < 0.5, residual=residual, scale=residual and rng.random() < 0.6,
                    pre=not post or rng.random() < 0.7, dtype=dtype)
    kv_heads, group = rng.choice([1, 2, 4, 6, 8]), rng.choice([1, 3, 4, 6, 8])
    width, page = rng.choice([64, 128, 128]), rng.choice([16, 48, 64, 128, 256])
    c = dict(op=kind, seqs=_log_int(rng, 1, 48), chunk=1, past=0, q_heads=kv_heads * group, kv_heads=kv_heads,
             width=width, page=page, dtype=dtype)
    if kind == "append":
        c["chunk"] = 1 if rng.random() < 0.3 else _log_int(rng, 2, 8192)
        c["seqs"] = max(1, min(c["seqs"], 32768 * 2 // (c["chunk"] * BYTES[dtype])))
        c["past"] = rng.choice([0, _log_int(rng, 1, 4096)])
        c["rot"] = rng.choice([width, width // 2])
        c["pairs"] = rng.random() < 0.5
        return c
    shape = rng.choice(["step", "draft", "chunk", "prompts"])
    if shape in ("step", "draft"):
        c["chunk"] = 1 if shape == "step" else rng.randint(2, 16)
        c["past"] = _log_int(rng, 16, 32767)
    else:
        c["chunk"] = _log_int(rng, 17, 2048)
        c["past"] = _log_int(rng, 16, 32767) if shape == "chunk" else 0
    if dtype == "f32":
        c["chunk"], c["past"] = min(c["chunk"], 512), min(c["past"], 8191)
    # at most the listed cases' cached values, and scores
    span = c["chunk"] + c["past"]
    c["seqs"] = max(1, min(c["seqs"], 32 * 8 * 32768 * 128 * 2 // (kv_heads * span * width * BYTES[dtype]),
                           16 * 2048 * 65536 // (c["q_heads"] * c["chunk"] * span)))
    return c


def _lengths(case):
    """(new tokens, past tokens) of each sequence: the last has the case's full sizes, the others from a
    sixteenth of them up, in a fixed mixed order; with one new token a step every sequence has one."""
    n, top, past = case["seqs"], case["chunk"], case["past"]
    share = [(1 + (5 * (n - 1 - b)) % n if math.gcd(5, n) == 1 else n - b) / n for b in range(n)]
    share = [1.0 if b == n - 1 else 1 / 16 + 15 / 16 * s for b, s in enumerate(share)]
    new = [top if top <= 16 or b == n - 1 else max(1, int(top * s)) for b, s in enumerate(share)]
    return new, [int(past * s) for s in share]


def _positions(case):
    new, past = _lengths(case)
    return sum(new), sum(new) + sum(past)


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] == "append":
        tokens, _ = _positions(case)
        values = tokens * case["width"] * (case["q_heads"] + 2 * case["kv_heads"])
        turned = tokens * case["rot"] * (case["q_heads"] + case["kv_heads"])
        return {"bytes": 2 * values * e + tokens * case["rot"] * 4, "flops": 3 * turned}
    if case["op"] == "attn":
        tokens, cached = _positions(case)
        new, past = _lengths(case)
        pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
        read = cached * case["kv_heads"] * 2 + tokens * case["q_heads"] * 2
        return {"bytes": read * case["width"] * e, "flops": 4 * pairs * case["q_heads"] * case["width"]}
    size = case["rows"] * case["groups"] * case["width"]
    ins = 1 + case["gate"] + case["residual"]
    outs = 1 + case["pre"]
    if not case["train"]:
        return {"bytes": (ins + outs) * size * e, "flops": 10 * size}
    return {"bytes": (2 * ins + 2 * outs) * size * e, "flops": 40 * size}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, mean=0.0, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std).add_(mean).to(dt)

    s = dict(case=dict(case))
    if case["op"] == "norm":
        shape = (case["rows"], case["groups"], case["width"])
        w = case["width"]
        s["x"] = normal(*shape, mean=0.05, std=1.3)
        s["gate"] = normal(*shape, std=1.5) if case["gate"] else None
        s["residual"] = normal(*shape, std=2.0) if case["residual"] else None
        s["w_post"] = normal(w, mean=1.0, std=0.1) if case["post"] else None
        s["res_scale"] = normal(w, mean=0.5, std=0.1) if case["scale"] else None
        s["w_pre"] = normal(w, mean=1.0, std=0.1) if case["pre"] else None
        if case["train"]:
            s["dh"] = normal(*shape, std=0.5)
            s["dy"] = normal(*shape) if case["pre"] else None
        return s

    new, past = _lengths(case)
    n, page, hk, hq, d = case["seqs"], case["page"], case["kv_heads"], case["q_heads"], case["width"]
    total = [a + b for a, b in zip(new, past)]
    used = [-(-t // page) for t in total]
    per_seq, count = max(used), sum(used) + 3
    order = torch.randperm(count, generator=gen, device="cuda").to(torch.int32)
    starts = torch.tensor([sum(used[:b]) for b in range(n)], device="cuda")
    col = torch.arange(per_seq, device="cuda")
    held = col[None, :] < torch.tensor(used, device="cuda")[:, None]
    at = (starts[:, None] + col[None, :]).clamp_(max=count - 1)
    s["page_table"] = torch.where(held, order[at], torch.full_like(order[at], -1))
    s["cu_seqlens"] = torch.tensor([sum(new[:b]) for b in range(n + 1)], dtype=torch.int32, device="cuda")
    s["kv_lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    s["max_q"], s["max_kv"] = max(new), max(total)
    s["k_cache"] = normal(count, hk, page, d)
    s["v_cache"] = normal(count, hk, page, d, mean=0.1)
    tokens = sum(new)
    if case["op"] == "append":
        # the rows of one fused projection: q, k and v are views of it
        qkv = normal(tokens, hq + 2 * hk, d)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        rate = 10000.0 ** (-torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64) * 2 / case["rot"])
        angle = torch.arange(s["max_kv"], device="cuda", dtype=torch.float64)[:, None] * rate[None, :]
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    else:
        s["q"] = normal(tokens, hq, d, std=1.5)
        s["scale"] = d ** -0.5
    return s


# ---------------------------------------------------------------- plain forms (32 bits)
def _token_places(s):
    """(sequence, index in it, position in the cache) of every new token."""
    cu, lens = s["cu_seqlens"].long(), s["kv_lens"].long()
    tok = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(cu, tok, right=True) - 1
    i = tok - cu[b]
    return b, i, lens[b] - (cu[b + 1] - cu[b]) + i


def _rotate(x, cos, sin, rot, pairs):
    x = x.float()
    head, rest = x[..., :rot], x[..., rot:]
    if pairs:
        a, b = head[..., 0::2], head[..., 1::2]
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
    c, n = cos[:, None, :], sin[:, None, :]
    u, v = a * c - b * n, b * c + a * n
    head = torch.stack((u, v), -1).flatten(-2) if pairs else torch.cat((u, v), -1)
    return torch.cat((head, rest), -1)


def _append_plain(s):
    case = s["case"]
    b, _, pos = _token_places(s)
    page = s["page_table"].long()[b, pos // case["page"]]
    row = pos % case["page"]
    cos, sin = s["cos"][pos], s["sin"][pos]
    s["k_cache"][page, :, row] = _rotate(s["k"], cos, sin, case["rot"], case["pairs"]).to(s["k"].dtype)
    s["v_cache"][page, :, row] = s["v"]
    q = _rotate(s["q"], cos, sin, case["rot"], case["pairs"]).to(s["q"].dtype)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attn_plain(s):
    case = s["case"]
    n, hk, d, mq, mk = case["seqs"], case["kv_heads"], case["width"], s["max_q"], s["max_kv"]
    g = case["q_heads"] // hk
    b, i, pos = _token_places(s)
    table = s["page_table"].long().clamp(min=0)

    def dense(cache):  # [n, hk, mk, d]
        c = cache[table].float().permute(0, 2, 1, 3, 4)
        return c.reshape(n, hk, -1, d)[:, :, :mk]

    q = torch.zeros(n, mq, hk, g, d, device="cuda")
    q[b, i] = s["q"].float().view(-1, hk, g, d)
    limit = torch.full((n, mq), -1, device="cuda")
    limit[b, i] = pos
    q = q.permute(0, 2, 1, 3, 4).reshape(n, hk, mq * g, d)
    seen = torch.arange(mk, device="cuda")[None, None, :] <= limit.repeat_interleave(g, 1)[:, :, None]
    x = torch.matmul(q, dense(s["k_cache"]).transpose(-1, -2)).mul_(s["scale"])
    x.masked_fill_(~seen[:, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp_()
    total = x.sum(-1, keepdim=True)
    held = torch.arange(mk, device="cuda")[None, :] < s["kv_lens"][:, None]
    v = dense(s["v_cache"]).masked_fill(~held[:, None, :, None], 0.0)
    o = torch.matmul(x, v) / torch.where(total == 0, torch.ones_like(total), total)
    o = o.view(n, hk, mq, g, d).permute(0, 2, 1, 3, 4)
    return o[b, i].reshape(-1, hk * g, d).to(s["q"].dtype)


def _norm_plain(s):
    case, dt = s["case"], s["x"].dtype
    x = s["x"].float()
    r1 = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n = x * r1 * s["w_post"].float() if case["post"] else x
    if case["gate"]:
        gate = s["gate"].float()
        sig = 1.0 / (1.0 + torch.exp(-gate))
        act = gate * sig
    m = n * act if case["gate"] else n
    scaled = m * s["res_scale"].float() if case["scale"] else m
    h = s["residual"].float() + scaled if case["residual"] else scaled
    out = {"h": h.to(dt)}
    if case["pre"]:
        r2 = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
        out["y"] = (h * r2 * s["w_pre"].float()).to(dt)
    if not case["train"]:
        return out
    dh = s["dh"].float()
    if case["pre"]:
        dy = s["dy"].float()
        out["dw_pre"] = (dy * h * r2).sum((0, 1)).to(dt)
        t = dy * s["w_pre"].float()
        dh = dh + r2 * (t - h * r2.square() * (t * h).mean(-1, keepdim=True))
    if case["residual"]:
        out["dresidual"] = dh.to(dt)
    dm = dh
    if case["scale"]:
        out["dres_scale"] = (dh * m).sum((0, 1)).to(dt)
        dm = dh * s["res_scale"].float()
    dn = dm
    if case["gate"]:
        out["dgate"] = (dm * n * sig * (1.0 + gate * (1.0 - sig))).to(dt)
        dn = dm * act
    dx = dn
    if case["post"]:
        out["dw_post"] = (dn * x * r1).sum((0, 1)).to(dt)
        t = dn * s["w_post"].float()
        dx = r1 * (t - x * r1.square() * (t * x).mean(-1, keepdim=True))
    out["dx"] = dx.to(dt)
    return out


# ---------------------------------------------------------------- the framework's calls
def _append_own(s):
    import gated_deltanet_gdn_gb300 as gdn

    q = gdn.gdn_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["cu_seqlens"], s["kv_lens"],
                          q=s["q"], cos=s["cos"], sin=s["sin"],
                          flags=gdn.GDN_FLAG_ROPE_PAIRS if s["case"]["pairs"] else 0)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attn_own(s):
    import gated_deltanet_gdn_gb300 as gdn

    return gdn.gdn_paged_attn(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["cu_seqlens"], s["kv_lens"],
                              s["scale"], max_q=s["max_q"], max_kv=s["max_kv"])


def _norm_own(s):
    import gated_deltanet_gdn_gb300 as gdn

    case = s["case"]
    parts = dict(gate=s["gate"], residual=s["residual"], w_post=s["w_post"], res_scale=s["res_scale"],
                 w_pre=s["w_pre"], eps=EPS)
    h, y, stats = gdn.gdn_block_norm_fwd(s["x"], **parts)
    out = {"h": h, "y": y} if case["pre"] else {"h": h}
    if case["train"]:
        grads = gdn.gdn_block_norm_bwd(s["x"], stats, s["dh"], s["dy"], **parts)
        out.update({k: v for k, v in grads.items() if v is not None})
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _append_own, "attn": _attn_own, "norm": _norm_own}[op](state)
    return {"append": _append_plain, "attn": _attn_plain, "norm": _norm_plain}[op](state)


# ---------------------------------------------------------------- 64 bits, from the definitions
def _exact_norm(s):
    """Each part by its definition; the gradients by reverse differentiation in 64 bits."""
    case = s["case"]
    leaf = {k: s[k].double().requires_grad_() for k in ("x", "gate", "residual", "w_post", "res_scale", "w_pre")
            if s[k] is not None}

    def rms(t, w):
        return t / torch.sqrt((t * t).sum(-1, keepdim=True) / t.shape[-1] + EPS) * w

    h = rms(leaf["x"], leaf["w_post"]) if case["post"] else leaf["x"] * 1.0
    if case["gate"]:
        h = h * leaf["gate"] * torch.sigmoid(leaf["gate"])
    if case["scale"]:
        h = h * leaf["res_scale"]
    if case["residual"]:
        h = h + leaf["residual"]
    out = {"h": h}
    loss = (h * s["dh"].double()).sum() if case["train"] else None
    if case["pre"]:
        out["y"] = rms(h, leaf["w_pre"])
        if case["train"]:
            loss = loss + (out["y"] * s["dy"].double()).sum()
    out = {k: v.detach() for k, v in out.items()}
    if case["train"]:
        grads = torch.autograd.grad(loss, list(leaf.values()))
        out.update({"d" + k: g for k, g in zip(leaf, grads)})
    return out


def _exact_append(s):
    """Token by token position: the rotation as a product of complex numbers."""
    case = s["case"]
    new, past = _lengths(case)
    rot, table = case["rot"], s["page_table"].tolist()
    spot = [(table[b][p // case["page"]], p % case["page"], p) for b in range(case["seqs"])
            for p in range(past[b], past[b] + new[b])]
    page, row, pos = (torch.tensor(v, device="cuda") for v in zip(*spot))
    phase = torch.complex(s["cos"].double()[pos], s["sin"].double()[pos])[:, None, :]

    def turn(x):
        x = x.double()
        first = x[..., 0:rot:2] if case["pairs"] else x[..., :rot // 2]
        second = x[..., 1:rot:2] if case["pairs"] else x[..., rot // 2:rot]
        z = torch.complex(first.contiguous(), second.contiguous()) * phase
        y = x.clone()
        if case["pairs"]:
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        else:
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        return y

    k, v = s["k_cache"].double(), s["v_cache"].double()
    k[page, :, row], v[page, :, row] = turn(s["k"]), s["v"].double()
    return {"q": turn(s["q"]), "k_cache": k, "v_cache": v}


def _exact_attn(s):
    """Sequence by sequence and head by head, over the keys of its own length."""
    case = s["case"]
    new, past = _lengths(case)
    page, g = case["page"], case["q_heads"] // case["kv_heads"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(case["seqs"]):
        total = new[b] + past[b]
        pages = s["page_table"][b, :-(-total // page)].long()
        pos = past[b] + torch.arange(new[b], device="cuda")
        hidden = torch.arange(total, device="cuda")[None, :] > pos[:, None]
        for j in range(case["kv_heads"]):
            k = s["k_cache"][pages, j].reshape(-1, case["width"])[:total].double()
            v = s["v_cache"][pages, j].reshape(-1, case["width"])[:total].double()
            q = s["q"][at:at + new[b], j * g:(j + 1) * g].double().transpose(0, 1)
            x = (q @ k.T * s["scale"]).masked_fill(hidden, float("-inf"))
            out[at:at + new[b], j * g:(j + 1) * g] = (torch.softmax(x, -1) @ v).transpose(0, 1)
        at += new[b]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "norm": _exact_norm}[case["op"]](s)
