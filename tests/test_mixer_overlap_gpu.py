"""Outputs on the memory of inputs: refused where the kernels would read what they have written, and right where they are
allowed: columns of one buffer, the scan's output on its own rows, final states on the initial ones."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn

pytestmark = pytest.mark.gpu
SILU, SOFT = gdn.GDN_FLAG_CONV_SILU, gdn.GDN_FLAG_DT_SOFTPLUS


def _refused(*calls):
    for i, call in enumerate(calls):
        with pytest.raises(gdn.GdnError, match="shares memory"):
            call()
            pytest.fail(f"call {i} was not refused")


def test_convolution():
    gen = torch.Generator(device="cuda").manual_seed(1)
    N, C = 50, 24
    buf = torch.randn(N + 4, 3 * C, generator=gen, device="cuda")
    x, w, cu = buf[:N, :C], torch.randn(C, 4, generator=gen, device="cuda"), torch.tensor([0, 20, N], dtype=torch.int32, device="cuda")
    pool = torch.zeros(3, 3, C, device="cuda")
    states = torch.zeros(9 * C, device="cuda")

    def f(x, **more):
        return gdn.gdn_causal_conv_fwd(x, w, cu_seqlens=cu, flags=SILU, **more)

    one = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    line = buf.view(-1)
    _refused(lambda: f(x, out=x), lambda: f(x, out=buf[3:N + 3, :C]), lambda: f(x, out=buf[:N, C - 1:2 * C - 1]),
             lambda: f(x, out=line[2 * C + 1:].as_strided((N, C), (3 * C, 1))),  # a column over the row's end
             lambda: f(line[:N * C].view(N, C), out=line[C:(N + 1) * C].view(N, C)), lambda: f(x, out=line[:N * C].view(N, C)),
             lambda: gdn.gdn_causal_conv_fwd(x.unsqueeze(0), w, out=x.unsqueeze(0)),
             lambda: f(x, state0=states[:6 * C].view(2, 3, C), state_final=states[3 * C:9 * C].view(2, 3, C)),
             lambda: f(line[:N * C].view(N, C), state_final=line[C:7 * C].view(2, 3, C)),
             lambda: gdn.gdn_causal_conv_fwd(x[:2], w, cu_seqlens=one, state_final=pool[:1], out=pool.view(-1)[C:3 * C].view(2, C)),
             lambda: gdn.gdn_causal_conv_fwd(x[:2], w, cu_seqlens=one, state0=pool[:1], out=pool.view(-1)[C:3 * C].view(2, C)),
             lambda: gdn.gdn_causal_conv_fwd(x[:2], w, cu_seqlens=one, out=w.view(-1)[:2 * C].view(2, C)))
    want, last = f(x.contiguous())
    got, _ = f(x, out=buf[:N, C:2 * C])  # columns of the same buffer
    assert torch.equal(got, want) and got.data_ptr() == buf[:, C:].data_ptr()
    got, last2 = f(x, state0=pool[:2], state_final=pool[:2])
    assert torch.equal(got, want) and torch.equal(last2, last) and last2.data_ptr() == pool.data_ptr()


@pytest.mark.parametrize("N,bound", [(50, None), (50, 1), (3000, None)])  # whole sequences, token by token, in chunks
def test_scan(N, bound):
    gen = torch.Generator(device="cuda").manual_seed(2)
    D, S = 32, 16
    cu = torch.tensor([0, 20, N], dtype=torch.int32, device="cuda")

    def inputs():
        g = torch.Generator(device="cuda").manual_seed(N)
        buf = torch.randn(N, 4 * D + 2 * S, generator=g, device="cuda")
        u, dt, z = (buf[:, i * D:(i + 1) * D] for i in range(3))
        B, C = (buf[:, 4 * D + i * S:4 * D + (i + 1) * S].unsqueeze(1) for i in range(2))
        return buf, dict(u=u, dt=dt, z=z, B=B, C=C)

    A, skip = -torch.rand(D, S, generator=gen, device="cuda"), torch.randn(D, generator=gen, device="cuda")
    h0 = torch.randn(3, D, S, generator=gen, device="cuda")

    def f(s, **more):
        return gdn.gdn_selective_scan_fwd(**s, A=A, D=skip, cu_seqlens=cu, max_q=bound, flags=SOFT, **more)

    buf, s = inputs()
    cut = {k: t[:N - 1] for k, t in s.items()}
    _refused(lambda: f(s, out=buf[:, 1:D + 1]), lambda: f(s, out=buf[:, 4 * D:5 * D]), lambda: f(s, out=buf[:, 3 * D + 1:4 * D + 1]),
             lambda: f(cut, out=buf[1:, :D]), lambda: f(s, out=buf.view(-1)[:N * D].view(N, D)), lambda: f(s, h0=h0[:2], h_final=h0[1:]),
             lambda: f(s, h_final=buf.view(-1)[:2 * D * S].view(2, D, S)))
    want, last, _ = f(s)
    for name in (None, "u", "dt", "z"):  # a column of its own, and in place
        buf, s = inputs()
        own = h0[:2].clone().zero_()
        y, h, _ = f(s, out=buf[:, 3 * D:4 * D] if name is None else s[name], h0=own, h_final=own)
        assert torch.equal(y, want) and torch.equal(h, last)
        rest = [k for k in ("u", "dt", "z", "B", "C") if k != name]
        assert all(torch.equal(s[k], inputs()[1][k]) for k in rest)
