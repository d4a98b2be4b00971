"""A hybrid stack: gated delta rule layers with a softmax attention layer between them, and state space
layers if wanted, run as a server does: a prompt in chunks, then token by token.

Every block is  norm -> projections -> mixer -> per-head gated norm -> projection -> scaled
residual,  and the step between two blocks (scaled residual and the next block's norm) is
one call. Rule layers carry a state, attention layers a paged cache, state space layers a state and the last
inputs of their convolution. The weights are random;
the check at the end is that the same tokens give the same activations however they are
split into calls.

    python examples/hybrid_stack.py
"""
from __future__ import annotations

import os
import sys
from typing import Dict, List, Optional

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_gdn_gb300 as gdn  # noqa: E402

PAGE = 64
STATES, TAPS = 16, 4  # of a state space layer


class HybridStack:
    """`layers` names each layer's mixer: "r" (gated delta rule), "a" (attention) or "s" (convolution and selective scan)."""

    def __init__(self, layers: str = "rrra", heads: int = 6, kv_heads: int = 2, width: int = 128, batch: int = 2,
                 max_tokens: int = 1024, seed: int = 0, device: str = "cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.layers, self.H, self.Hk, self.D, self.B = layers, heads, kv_heads, width, batch
        self.model = heads * width
        self.device, self.dtype = device, torch.bfloat16

        def normal(*shape, std=None):
            std = shape[0] ** -0.5 if std is None else std
            return (torch.randn(*shape, generator=g, device=device) * std).to(self.dtype)

        self.weights: List[Dict[str, torch.Tensor]] = []
        for kind in layers:
            qkv = {"r": 3 * heads, "a": heads + 2 * kv_heads, "s": heads}[kind] * width
            w = {"qkv": normal(self.model, qkv), "gate": normal(self.model, self.model), "out": normal(self.model, self.model),
                 "pre": 1 + normal(self.model, std=0.1), "post": 1 + normal(width, std=0.1),
                 "scale": 0.5 + normal(self.model, std=0.1)}
            if kind == "r":
                w["g"], w["beta"] = normal(self.model, heads), normal(self.model, heads)
            elif kind == "s":
                w["conv"], w["bc"] = normal(self.model, TAPS, std=TAPS ** -0.5), normal(self.model, 2 * STATES)
                w["dt"], w["dt_bias"] = normal(self.model, self.model), torch.full((self.model,), -4.0, device=device)
                w["A"] = -torch.arange(1.0, STATES + 1, device=device).repeat(self.model, 1)
                w["D"] = torch.ones(self.model, device=device)
            self.weights.append(w)
        self.last_norm = 1 + normal(self.model, std=0.1)
        rate = 10000.0 ** (-torch.arange(width // 2, device=device, dtype=torch.float64) * 2 / width)
        angle = torch.arange(max_tokens, device=device, dtype=torch.float64)[:, None] * rate
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        self.pages = -(-max_tokens // PAGE)
        self.reset()

    def reset(self) -> None:
        """Empty states and caches (cache rows hold nothing until they are appended)."""
        B, H, D = self.B, self.H, self.D
        self.states = [torch.zeros(B, H, D, D, device=self.device) if k == "r" else
                       torch.zeros(B, self.model, STATES, device=self.device) if k == "s" else None for k in self.layers]
        self.inputs = [torch.zeros(B, TAPS - 1, self.model, dtype=self.dtype, device=self.device) if k == "s" else None
                       for k in self.layers]
        shape = (B * self.pages, self.Hk, PAGE, D)
        self.caches = [[torch.empty(shape, dtype=self.dtype, device=self.device) for _ in range(2)] if k == "a" else None
                       for k in self.layers]
        order = torch.randperm(B * self.pages, device=self.device).to(torch.int32)
        self.page_table = order.view(B, self.pages)
        self.kv_lens = torch.zeros(B, dtype=torch.int32, device=self.device)
        self.length = 0

    def _rule(self, i: int, y: torch.Tensor, w) -> torch.Tensor:
        B, T = y.shape[:2]
        q, k, v = (y @ w["qkv"]).view(B, T, 3, self.H, self.D).unbind(2)
        g = torch.nn.functional.logsigmoid((y @ w["g"]).float() + 2.0).to(self.dtype)
        beta = torch.sigmoid(y @ w["beta"])
        out, _ = gdn.gdn_recurrent(q.contiguous(), k.contiguous(), v.contiguous(), g, beta, self.states[i],
                                   h_final=self.states[i], flags=gdn.GDN_FLAG_QK_L2NORM)
        return out

    def _attention(self, i: int, y: torch.Tensor, w) -> torch.Tensor:
        B, T = y.shape[:2]
        kc, vc = self.caches[i]
        qkv = (y @ w["qkv"]).view(B * T, self.H + 2 * self.Hk, self.D)
        q, k, v = qkv[:, :self.H], qkv[:, self.H:self.H + self.Hk], qkv[:, self.H + self.Hk:]
        where = (kc, vc, self.page_table, self.cu_seqlens, self.kv_lens)
        q = gdn.gdn_kv_append(k, v, *where, q=q, cos=self.cos, sin=self.sin)
        return gdn.gdn_paged_attn(q, *where, max_q=T, max_kv=self.length).view(B, T, self.H, self.D)

    def _state_space(self, i: int, y: torch.Tensor, w) -> torch.Tensor:
        B, T = y.shape[:2]
        u, _ = gdn.gdn_causal_conv_fwd(y @ w["qkv"], w["conv"], state0=self.inputs[i], state_final=self.inputs[i],
                                       flags=gdn.GDN_FLAG_CONV_SILU)
        Bm, Cm = (t.unflatten(-1, (1, STATES)) for t in (u @ w["bc"]).split(STATES, -1))
        out, _, _ = gdn.gdn_selective_scan_fwd(u, u @ w["dt"], w["A"], Bm, Cm, D=w["D"], dt_bias=w["dt_bias"], h0=self.states[i],
                                               h_final=self.states[i], flags=gdn.GDN_FLAG_DT_SOFTPLUS)
        return out.view(B, T, self.H, self.D)

    def step(self, x: torch.Tensor) -> torch.Tensor:
        """Next T tokens' activations x [B, T, model] -> the stack's normed output, same shape."""
        B, T = x.shape[:2]
        self.length += T
        self.kv_lens += T
        self.cu_seqlens = torch.arange(B + 1, dtype=torch.int32, device=self.device) * T
        h, y, _ = gdn.gdn_block_norm_fwd(x.reshape(B * T, self.model), w_pre=self.weights[0]["pre"])
        for i, w in enumerate(self.weights):
            y = y.view(B, T, self.model)
            mixed = {"r": self._rule, "a": self._attention, "s": self._state_space}[self.layers[i]](i, y, w)
            gate = (y @ w["gate"]).view(B, T, self.H, self.D)
            o, _, _ = gdn.gdn_block_norm_fwd(mixed, gate=gate, w_post=w["post"])
            block = o.view(B * T, self.model) @ w["out"]
            after = self.weights[i + 1]["pre"] if i + 1 < len(self.weights) else self.last_norm
            h, y, _ = gdn.gdn_block_norm_fwd(block, residual=h, res_scale=w["scale"], w_pre=after)
        return y.view(B, T, self.model)


def run(tokens: int = 300, prompt: int = 200, chunk: int = 128, stack: Optional[HybridStack] = None, seed: int = 1):
    """(whole, parts): the outputs of all tokens in one call, and of the same tokens as a prompt in
    chunks followed by single tokens."""
    s = stack or HybridStack()
    g = torch.Generator(device=s.device).manual_seed(seed)
    x = torch.randn(s.B, tokens, s.model, generator=g, device=s.device).to(s.dtype)
    whole = s.step(x)
    s.reset()
    parts, at = [], 0
    while at < tokens:
        n = min(chunk, prompt - at) if at < prompt else 1
        parts.append(s.step(x[:, at:at + n]))
        at += n
    return whole, torch.cat(parts, 1)


if __name__ == "__main__":
    whole, parts = run()
    d = (whole.double() - parts.double()).norm() / whole.double().norm()
    print(f"300 tokens at once against 200 in chunks and 100 one by one: relative difference {float(d):.2e}")
    assert float(d) < 2e-2 and gdn.gdn_check_device_error() == gdn.binding.GDN_OK
