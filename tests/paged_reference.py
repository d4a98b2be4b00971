"""Paged cache cases and their plain float64 forms, on the CPU, written from the formulas
in include/gdn.h (no code shared with the kernels)."""
from __future__ import annotations

import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# relative size of one rounding to the type: half the distance between neighbours
UNIT = {k: torch.finfo(t).eps / 2 for k, t in DT.items()}


class Paged:
    """Sequences with new[b] new tokens and length[b] cached tokens (new ones included) in
    shuffled pages. Everything that no token owns is NaN: rows past a length, spare pages.
    rows_first: the cache's memory is [page, row, head, channel] instead of [page, head, row, channel]."""

    def __init__(self, new, length, Hq, Hk, D, page, dtype, seed=0, rows_first=False, fill=True, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.new, self.length, self.Hq, self.Hk, self.D, self.page = list(new), list(length), Hq, Hk, D, page
        self.dtype, self.dt = dtype, DT[dtype]
        B = len(new)
        used = [-(-max(n, 0) // page) for n in length]
        self.per = max(max(used), 1) + 1
        self.count = sum(used) + spare
        order = torch.randperm(self.count, generator=g).tolist()
        self.table = torch.full((B, self.per), -1, dtype=torch.int32)
        self.kc = torch.full((self.count, Hk, page, D), float("nan"), dtype=self.dt)
        self.vc = self.kc.clone()
        at = 0
        for b in range(B):
            for i in range(used[b]):
                pg = order[at]
                at += 1
                self.table[b, i] = pg
                held = min(page, length[b] - i * page)
                if fill:
                    self.kc[pg, :, :held] = torch.randn(Hk, held, D, generator=g).to(self.dt)
                    self.vc[pg, :, :held] = (torch.randn(Hk, held, D, generator=g) + 0.1).to(self.dt)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        self.lens = torch.tensor(length, dtype=torch.int32)
        self.N = int(sum(new))
        self.g = g
        self.rows_first = rows_first

    def normal(self, *shape, std=1.0):
        return (torch.randn(*shape, generator=self.g) * std).to(self.dt)

    def cuda(self):
        """(k_cache, v_cache, page_table, cu_seqlens, kv_lens) on the GPU."""
        if self.rows_first:
            kc, vc = (c.transpose(1, 2).contiguous().cuda().transpose(1, 2) for c in (self.kc, self.vc))
        else:
            kc, vc = self.kc.cuda(), self.vc.cuda()
        return kc, vc, self.table.cuda(), self.cu.cuda(), self.lens.cuda()

    def tokens(self):
        """(token, sequence, position) of every new token."""
        return [(int(self.cu[b]) + i, b, self.length[b] - n + i) for b, n in enumerate(self.new) for i in range(n)]

    def dense(self, cache, b):
        """[Hk, length, D] float64 of sequence b."""
        n = self.length[b]
        pages = self.table[b, :-(-n // self.page)].long()
        c = cache[pages].double()  # [pages, Hk, page, D]
        return c.permute(1, 0, 2, 3).reshape(self.Hk, -1, self.D)[:, :n]


def attention(c: Paged, q: torch.Tensor, scale: float):
    """(out, |.|-weighted out, lse, largest sum |q k| scale) in float64; rows without keys are 0 and -inf."""
    N, Hq, D = q.shape
    out = torch.zeros(N, Hq, D, dtype=torch.float64)
    mag, lse = torch.zeros_like(out), torch.full((N, Hq), -float("inf"), dtype=torch.float64)
    G, size = Hq // c.Hk, 0.0
    for b, n in enumerate(c.new):
        if n == 0 or c.length[b] <= 0:
            continue
        K, V = c.dense(c.kc, b), c.dense(c.vc, b)
        t0 = int(c.cu[b])
        qb = q[t0:t0 + n].double().reshape(n, c.Hk, G, D)
        s = torch.einsum("nhgd,hkd->nhgk", qb, K) * scale
        size = max(size, float((torch.einsum("nhgd,hkd->nhgk", qb.abs(), K.abs()) * scale).max()))
        pos = c.length[b] - n + torch.arange(n)
        seen = torch.arange(K.shape[1])[None, :] <= pos[:, None]
        for i in range(n):
            if int(pos[i]) < 0:
                continue
            k = int(pos[i]) + 1
            si = s[i, :, :, :k]
            l = torch.logsumexp(si, -1)
            p = torch.exp(si - l[..., None])
            out[t0 + i] = torch.einsum("hgk,hkd->hgd", p, V[:, :k]).reshape(Hq, D)
            mag[t0 + i] = torch.einsum("hgk,hkd->hgd", p, V[:, :k].abs()).reshape(Hq, D)
            lse[t0 + i] = l.reshape(Hq)
        del seen
    return out, mag, lse, size


def attention_bounds(c: Paged, out, mag, lse, size):
    """Error bounds of the kernels, element by element. Scores: products in the inputs' type accumulate
    in fp32 (fp32: three TF32 terms), off by at most 2^-19 of sum |q k|, which moves a probability by
    that much relatively, and its normalised sum alike; the second product and its sum add 2^-18 and one
    fp32 rounding per key. bf16 rounds each probability and the result once."""
    keys = max(max(c.length), 1)
    fp32 = 2.0 ** -18 * (1 + size) + keys * 2.0 ** -24
    tol = mag * fp32 + out.abs() * UNIT[c.dtype]
    if c.dtype == "bf16":
        tol = tol + mag * UNIT["bf16"]
    finite = torch.where(torch.isinf(lse), torch.zeros_like(lse), lse).abs()
    return tol + 1e-30, 2.0 ** -19 * (1 + size) + finite * 2.0 ** -21 + keys * 2.0 ** -24


def rotated(x: torch.Tensor, pos, cos, sin, pairs: bool):
    """(float64 rotated [tokens, heads, D], |a| + |b| of each element's pair)."""
    rot = 2 * cos.shape[1]
    y = x.double().clone()
    mag = x.double().abs()
    i = torch.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
    c, s = cos.double()[pos][:, None], sin.double()[pos][:, None]
    a, b = x.double()[..., ia], x.double()[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return y, mag
