"""The causal convolution, the selective scan and the plan of a step in 64 bits, from their definitions, sequence by
sequence, with bounds of what float32 arithmetic may be off."""
import torch

# Relative error of one step of the kernels' float32 arithmetic: the approximate exponential and reciprocal are within
# 2^-22, softplus (both, and a series) within 2^-21, products and sums add 2^-24 each; a handful of them stay below 2^-20.
UNIT = 2.0 ** -20


def within(name, got, want, bound):
    """Every element within its bound and one rounding (half a step) to the output's type."""
    assert got.shape == want.shape, (name, got.shape, want.shape)
    half = torch.finfo(got.dtype).eps / 2
    off = (got.double() - want).abs()
    room = half * (want.abs() + bound) + bound + 1e-37
    assert bool(torch.isfinite(got.double()).all()), name
    worst = float((off / room).max()) if off.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.2f} times its bound"


def conv_seq(x, w, bias, state, silu, dy=None, dstate=None):
    """One sequence [T, C]: {name: (value, bound)}. Gradients by reverse differentiation."""
    k, T = w.shape[1], x.shape[0]
    x, w, state = (t.detach().double().requires_grad_() for t in (x, w, state))
    b = (torch.zeros(x.shape[1], dtype=torch.float64, device=x.device) if bias is None else bias.detach().double()).requires_grad_()
    seq = torch.cat((state, x))
    pre = sum(seq[j:j + T] * w[:, j] for j in range(k)) + b
    size = (sum(seq[j:j + T].abs() * w[:, j].abs() for j in range(k)) + b.abs()).detach()
    y = pre * torch.sigmoid(pre) if silu else pre * 1.0
    # silu' is at most 1.1, and its own error relative to |y| (1 + |pre|)
    bound = UNIT * (2 * size + y.detach().abs() * (1 + pre.detach().abs()))
    out = {"y": (y.detach(), bound), "state": (seq[T:].detach(), torch.zeros_like(seq[T:]))}
    if dy is None:
        return out
    loss = (y * dy.double()).sum()
    if dstate is not None:
        loss = loss + (seq[T:] * dstate.double()).sum()
    g = torch.autograd.grad(loss, (x, w, b, state))
    # |silu''| is at most 0.5: what pre is off moves dpre by half of that; then sums over taps, or over T tokens
    dpre = dy.double().abs() * (1.1 if silu else 1.0)
    off = UNIT * dy.double().abs() * (1.0 + size + pre.detach().abs()) if silu else torch.zeros_like(dpre)
    reach = torch.zeros(T + k - 1, x.shape[1], dtype=torch.float64, device=x.device)
    for j in range(k):
        reach[j:j + T] += w[:, j].detach().abs() * (off + UNIT * dpre)
    if dstate is not None:
        reach[T:] += UNIT * dstate.double().abs()
    many = UNIT + T * 2.0 ** -24
    a = seq.detach().abs()
    dw = torch.stack([(a[j:j + T] * (off + many * dpre)).sum(0) for j in range(k)], 1)
    out.update(dx=(g[0], reach[k - 1:]), dweight=(g[1], dw), dbias=(g[2], (off + many * dpre).sum(0)),
               dstate0=(g[3], reach[:k - 1]))
    return out


def scan_seq(u, dt, A, B, C, D=None, z=None, bias=None, softplus=True, h0=None, dy=None, dh=None):
    """One sequence, u, dt, z [T, D], B, C [T, G, S]: {name: (value, bound)}, token by token. Beside each value runs the
    sum of its terms' magnitudes, and the error a step adds to it."""
    T, d = u.shape
    s = A.shape[1]
    like = dict(dtype=torch.float64, device=u.device)
    u, raw, A = u.double(), dt.double() + (0 if bias is None else bias.double()), A.double()
    skip = torch.zeros(d, **like) if D is None else D.double()
    B, C = (t.double().repeat_interleave(d // t.shape[1], 1) for t in (B, C))
    step = torch.nn.functional.softplus(raw, threshold=700.0) if softplus else raw
    a = torch.exp(step[:, :, None] * A)
    grow = UNIT * (1 + 4 * (step[:, :, None] * A).abs())
    x = (step * u)[:, :, None] * B
    h = torch.zeros(d, s, **like) if h0 is None else h0.double()
    hb, e = h.abs(), torch.zeros(d, s, **like)
    hs, hbs, es = [h], [hb], [e]
    for t in range(T):
        h, hb = a[t] * h + x[t], a[t] * hb + x[t].abs()
        e = a[t] * e + grow[t] * hb
        hs.append(h), hbs.append(hb), es.append(e)
    H, HB, E = (torch.stack(v) for v in (hs, hbs, es))
    y0 = (C * H[1:]).sum(-1) + skip * u
    yb = (C.abs() * HB[1:]).sum(-1) + (skip * u).abs()
    ye = (C.abs() * E[1:]).sum(-1) + UNIT * yb
    gate, gs, zd = torch.ones_like(u), torch.zeros_like(u), torch.zeros_like(u)
    if z is not None:
        zd = z.double()
        sg = torch.sigmoid(zd)
        gate, gs = zd * sg, sg * (1 + zd * (1 - sg))
    soft = UNIT * (1 + zd.abs())  # of the gate and its slope
    out = {"y": (y0 * gate, gate.abs() * (ye + soft * yb)), "h": (h, e)}
    if dy is None:
        return out
    dy = dy.double()
    dg = dy * gate
    carry = torch.zeros(d, s, **like) if dh is None else dh.double()
    cb, ce = carry.abs(), torch.zeros(d, s, **like)
    G, GB, GE = (torch.zeros(T, d, s, **like) for _ in range(3))
    for t in range(T - 1, -1, -1):
        own = C[t] * dg[t][:, None]
        G[t], GB[t] = own + carry, own.abs() + cb
        GE[t] = ce + (UNIT + soft[t])[:, None] * GB[t]
        carry, cb = a[t] * G[t], a[t] * GB[t]
        ce = a[t] * GE[t] + grow[t] * cb
    t1, tb = G * a * H[:-1], GB * a * HB[:-1]
    te = GE * a * HB[:-1] + GB * a * E[:-1] + grow * tb
    many = UNIT + T * 2.0 ** -24
    gx, gxe = (G * B).sum(-1), ((GE + UNIT * GB) * B.abs()).sum(-1)
    gxb = (GB * B.abs()).sum(-1)
    gd, gde = (t1 * A).sum(-1), ((te + UNIT * tb) * A.abs()).sum(-1)
    gdb = (tb * A.abs()).sum(-1)
    slope = torch.sigmoid(raw) if softplus else torch.ones_like(raw)
    ddt = (gd + gx * u) * slope
    ddte = (gde + gxe * u.abs() + UNIT * (2 + raw.abs()) * (gdb + gxb * u.abs())) * slope
    out["ddt"] = (ddt, ddte)
    out["du"] = (gx * step + dg * skip, gxe * step.abs() + UNIT * (gxb * step.abs()) + (UNIT + soft) * (dg * skip).abs())
    out["dz"] = (dy * y0 * gs, dy.abs() * (1.1 * ye + 2 * soft * yb))
    per = (T, C.shape[2])
    out["dB"] = (G * (step * u)[:, :, None], (GE + 2 * UNIT * GB) * (step * u)[:, :, None].abs())
    out["dC"] = (H[1:] * dg[:, :, None], (E[1:] + (2 * UNIT + soft[:, :, None]) * HB[1:]) * dg[:, :, None].abs())
    out["dA"] = ((t1 * step[:, :, None]).sum(0), ((te + many * tb) * step[:, :, None].abs()).sum(0))
    out["dD"] = ((dg * u).sum(0), ((many + soft) * (dg * u).abs()).sum(0))
    out["ddt_bias"] = (ddt.sum(0), (ddte + many * (gdb + gxb * u.abs()) * slope).sum(0))
    out["dh0"] = (carry, ce)
    assert per[1] == s
    return out


def over_channels(pair, groups):
    """Values and bounds [T, D, S] summed over each group's channels."""
    v, b = pair
    T, d, s = v.shape
    many = d * 2.0 ** -24
    return tuple(t.reshape(T, groups, d // groups, s).sum(2) for t in (v, b + many * v.abs()))


def plan(table, lens, new, free, count, page, top):
    """The plan of a step with lists: request by request, a list for the stack. Changes nothing it is given."""
    table, slots, n = [list(r) for r in table], list(free), len(lens)
    cap = (len(table[0]) if n else 0) * page
    stack = slots[:count]
    lens = [min(max(v, 0), cap) for v in lens]
    kept = list(lens)
    for b in range(n):
        if new[b] < 0:
            kept[b] = max(0, lens[b] + new[b])
            stack += table[b][-(-kept[b] // page):-(-lens[b] // page)]
    slots[count:] = (stack[count:] + slots[len(stack):])[:len(slots) - count]
    have, asked, tokens, cu, rows = len(stack), 0, 0, [0], []
    for b in range(n):
        ask = new[b] if 0 < new[b] <= cap - lens[b] else 0
        pages = -(-(lens[b] + ask) // page) - -(-lens[b] // page) if ask else 0
        asked, tokens = asked + pages, tokens + ask
        if (pages and asked > have) or tokens > top:
            ask = pages = 0
        for j in range(pages):
            table[b][-(-lens[b] // page) + j] = stack.pop()
        rows += [(b, p, table[b][p // page] * page + p % page) for p in range(lens[b], lens[b] + ask)]
        kept[b] += ask
        cu.append(len(rows))
    rows += [(-1, -1, -1)] * (top - len(rows))
    r, p, s = (list(v) for v in zip(*rows)) if rows else ([], [], [])
    return dict(cu_seqlens=cu, kv_lens=kept, free_count=[min(len(stack), len(slots))], requests=r, positions=p, slots=s,
                page_table=table, free_pages=slots)
