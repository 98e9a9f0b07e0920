"""The mixer's operators as they are used together: in-proj columns through the
convolution, the scan and the gated norm, for a prompt and then single tokens."""
import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from tests import mixer_ref as ref

pytestmark = pytest.mark.gpu

H, P, G, N, TAPS, EPS = 6, 80, 2, 128, 4, 1e-5
INNER, CD = H * P, H * P + 2 * G * N
GROUP = INNER // G


class Mixer:
    def __init__(self, rows, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.inproj = torch.randn(rows, INNER + CD + H, generator=gen).to(torch.bfloat16).cuda()
        self.w = (torch.randn(CD, TAPS, generator=gen) / 2).cuda()
        self.bias = (0.1 * torch.randn(CD, generator=gen)).cuda()
        self.a = -(1 + 15 * torch.rand(H, generator=gen)).cuda()
        self.d = torch.randn(H, generator=gen).cuda()
        self.dt_bias = (torch.randn(H, generator=gen) - 3).cuda()
        self.norm_w = (1 + 0.1 * torch.randn(INNER, generator=gen)).cuda()

    def split(self, rows):
        p = self.inproj[rows]
        return p[:, :INNER], p[:, INNER:INNER + CD], p[:, INNER + CD:]

    def prompt(self, rows, conv_state, ssm_state, cu, slots, resume):
        z, u, dt = self.split(rows)
        xbc = g.causal_conv(u, self.w, self.bias, cu_seqlens=cu, state=conv_state, slots=slots,
                            resume=resume)
        y = g.ssm_scan(xbc[:, :INNER], dt, self.a, xbc[:, INNER:INNER + G * N],
                       xbc[:, INNER + G * N:], head_dim=P, state_size=N, d=self.d,
                       dt_bias=self.dt_bias, cu_seqlens=cu, state=ssm_state, slots=slots,
                       resume=resume)
        return xbc, y, g.forward(y, z, self.norm_w, group_size=GROUP, eps=EPS)

    def reference(self, spans, xbc, y):
        """Each stage's reference from the previous stage's actual output."""
        z, u, dt = (t.float().cpu() for t in self.split(slice(None)))
        want_x, bound_x, _ = ref.conv(u, self.w, self.bias, spans=spans)
        x = xbc.cpu()
        want_y, bound_y, size, *_ = ref.scan(x[:, :INNER], dt, self.a, x[:, INNER:INNER + G * N],
                                             x[:, INNER + G * N:], P, N, self.d, self.dt_bias,
                                             spans=spans)
        v = y.double().cpu() * (z.double() * torch.sigmoid(z.double()))
        v = v.reshape(-1, G, GROUP)
        n = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
        return want_x, bound_x, want_y, bound_y, size, n.reshape(-1, INNER) * self.norm_w.double().cpu()


def _check(m, spans, xbc, y, out):
    want_x, bound_x, want_y, bound_y, size, want_o = m.reference(spans, xbc, y)
    half = torch.finfo(torch.bfloat16).eps / 2
    f = lambda t: t.double().cpu()  # noqa: E731
    slack = 1 + 2.0 ** -6
    assert ((f(xbc) - want_x).abs() <= bound_x + ref.rounding(want_x, torch.bfloat16) * slack).all()
    assert ((f(y) - want_y).abs() <= (bound_y + ref.rounding(want_y, torch.bfloat16) + size * half)
            * slack).all()
    # the norm rounds twice
    assert ((f(out) - want_o).abs() <= want_o.abs() * 2 * half * slack + 1e-30).all()


def test_prompts_then_tokens():
    """Two ragged prompts, then tokens one by one from their states (eagerly for
    one, in a replayed graph for the next): as if each had come at once."""
    total, more = (130, 37), 5
    rows = sum(total)
    m = Mixer(rows)
    conv_state = torch.full((4, TAPS - 1, CD), 9.0, dtype=torch.bfloat16, device="cuda")
    ssm_state = torch.full((4, H, P, N), 9.0, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    fresh = torch.zeros(2, dtype=torch.bool, device="cuda")
    heads = [list(range(0, total[0] - more)), list(range(total[0], rows - more))]
    cu = torch.tensor([0, len(heads[0]), len(heads[0]) + len(heads[1])], dtype=torch.int32).cuda()
    index = torch.tensor(heads[0] + heads[1], device="cuda")
    got = [torch.empty(rows, n, dtype=torch.bfloat16, device="cuda") for n in (CD, INNER, INNER)]
    for into, part in zip(got, m.prompt(index, conv_state, ssm_state, cu, slots, fresh)):
        into[index] = part
    # decode: static buffers, the three calls captured in one graph
    buf = torch.empty(2, INNER + CD + H, dtype=torch.bfloat16, device="cuda")
    xbc = torch.empty(2, CD, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(2, INNER, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(y)
    steps = [dict(op="causal_conv_step", x=buf[:, INNER:INNER + CD], state=conv_state, weight=m.w,
                  bias=m.bias, slots=slots, out=xbc),
             dict(op="ssm_scan_step", x=xbc[:, :INNER], dt=buf[:, INNER + CD:], a=m.a,
                  b=xbc[:, INNER:INNER + G * N], c=xbc[:, INNER + G * N:], state=ssm_state, d=m.d,
                  dt_bias=m.dt_bias, slots=slots, out=y),
             dict(y=y, gate=buf[:, :INNER], w=m.norm_w, out=out, group_size=GROUP, eps=EPS)]
    graph = g.DecodeGraph(steps)
    single = [g.DecodeGraph([s]) for s in steps]
    for t in range(more):
        at = torch.tensor([total[0] - more + t, rows - more + t], device="cuda")
        buf.copy_(m.inproj[at])
        if t == 0:
            g.causal_conv_step(buf[:, INNER:INNER + CD], conv_state, m.w, m.bias, slots=slots,
                               out=xbc)
            g.ssm_scan_step(xbc[:, :INNER], buf[:, INNER + CD:], m.a, xbc[:, INNER:INNER + G * N],
                            xbc[:, INNER + G * N:], ssm_state, d=m.d, dt_bias=m.dt_bias,
                            slots=slots, out=y)
            g.forward(y, buf[:, :INNER], m.norm_w, group_size=GROUP, eps=EPS, out=out)
        elif t == 1:
            for one in single:
                one.replay()
        else:
            graph.replay()
        for into, part in zip(got, (xbc, y, out)):
            into[at] = part
    torch.cuda.synchronize()
    _check(m, [(0, total[0]), (total[0], rows)], *got)
    # entries of no sequence are as they were
    assert (conv_state[[0, 2]] == 9.0).all() and (ssm_state[[0, 2]] == 9.0).all()


def test_a_graph_refuses_what_it_does_not_know():
    with pytest.raises(ValueError, match="unknown op"):
        g.DecodeGraph([dict(op="conv")])
    x = torch.zeros(1, 8, device="cuda")
    st, w = torch.zeros(1, 3, 8, device="cuda"), torch.zeros(8, 4, device="cuda")
    with pytest.raises(ValueError, match="needs out"):
        g.DecodeGraph([dict(op="causal_conv_step", x=x, state=st, weight=w)])
    with pytest.raises(ValueError, match="takes no"):
        g.DecodeGraph([dict(op="causal_conv_step", x=x, state=st, weight=w, out=torch.zeros_like(x),
                            resume=None)])
