"""Layer norm, recurrence and gated norm as a layer uses them together: a training
step forward and backward, decoding in a graph, calls of several threads, tensors
past 2^31 elements, and what the binding refuses."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from tests import train_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
T = torch.bfloat16
MODEL, WIDTH, GROUP, EPS = 192, 320, 80, 1e-5
CU = [0, 1, 130, 130, 400]
SPANS = list(zip(CU[:-1], CU[1:]))


class Layer:
    """x -> layer norm -> projection -> [x | input gate | decay gate | z] -> recurrence ->
    gated norm with z -> projection."""

    def __init__(self, rows, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.x = (torch.randn(rows, MODEL, generator=gen) + 0.3).to(T).cuda()
        self.w = (1 + 0.1 * torch.randn(MODEL, generator=gen)).cuda()
        self.b = (0.1 * torch.randn(MODEL, generator=gen)).cuda()
        self.w_in = (torch.randn(4 * WIDTH, MODEL, generator=gen) / MODEL ** 0.5).to(T).cuda()
        self.a = (-0.1 * torch.rand(WIDTH, generator=gen)).cuda()
        self.norm_w = (1 + 0.1 * torch.randn(WIDTH, generator=gen)).cuda()
        self.w_out = (torch.randn(MODEL, WIDTH, generator=gen) / WIDTH ** 0.5).to(T).cuda()
        self.dout = torch.randn(rows, MODEL, generator=gen).to(T).cuda()

    @staticmethod
    def columns(t):
        return [t[:, k * WIDTH:(k + 1) * WIDTH] for k in range(4)]

    def forward(self, cu):
        xn = g.layer_norm(self.x, self.w, self.b, eps=EPS)
        proj = xn @ self.w_in.t()
        u, i, r, z = self.columns(proj)
        saved = g.linear_recurrence_saved(u)
        y = g.linear_recurrence(u, i, r, self.a, cu_seqlens=cu, saved=saved)
        return xn, proj, saved, y, g.forward(y, z, self.norm_w, group_size=GROUP, eps=EPS)

    def backward(self, cu, xn, proj, saved, y, h):
        u, i, r, z = self.columns(proj)
        dproj = torch.empty_like(proj)
        du, di, dr, dz = self.columns(dproj)
        dh = self.dout @ self.w_out
        dy, _, dnorm = g.backward(dh, y, z, self.norm_w, group_size=GROUP, eps=EPS, dgate=dz)
        _, _, _, da, _ = g.linear_recurrence_backward(dy, u, i, r, self.a, cu_seqlens=cu,
                                                      saved=saved, dx=du, dinput_gate=di,
                                                      ddecay_gate=dr)
        dxn = dproj @ self.w_in
        dx, dw, db = g.layer_norm_backward(dxn, self.x, self.w, eps=EPS)
        return dh, dy, dz, dnorm, dproj, da, dxn, dx, dw, db

    def step(self, cu):
        kept = self.forward(cu)
        return kept + self.backward(cu, *kept)


def test_a_training_step():
    """Each stage against its formulas in 64 bits from the previous stage's output."""
    m = Layer(CU[-1])
    xn, proj, saved, y, h, dh, dy, dz, dnorm, dproj, da, dxn, dx, dw, db = m.step(
        torch.tensor(CU, dtype=torch.int32).cuda())
    u, i, r, z = m.columns(proj)
    ref.assert_close(xn, *ref.layer_norm(m.x, m.w, m.b, EPS), T, "layer norm")
    want, bound, *_ = ref.recur(u, i, r, m.a, SPANS)
    ref.assert_close(y, want, bound, T, "recurrence")
    want = ref.norm_backward(dh, y, z, m.norm_w, GROUP, EPS, "mamba2")
    for n, v in (("dy", dy), ("dgate", dz), ("dw", dnorm)):
        ref.assert_close(v, *want[n], torch.float32 if n == "dw" else T, n)
    want = ref.recur_backward(dy, u, i, r, m.a, SPANS)
    du, di, dr, _ = m.columns(dproj)
    for n, v in (("dx", du), ("di", di), ("dr", dr), ("da", da)):
        ref.assert_close(v, *want[n], torch.float32 if n == "da" else T, n)
    want = ref.layer_norm_backward(dxn, m.x, m.w, EPS)
    for n, v in (("dx", dx), ("dw", dw), ("db", db)):
        ref.assert_close(v, *want[n], T if n == "dx" else torch.float32, n)


def test_the_gradients_are_those_of_the_whole_layer():
    """Against torch's differentiation of the layer in 64 bits: the gradient's direction
    and size (16-bit roundings between stages)."""
    m = Layer(CU[-1], seed=1)
    got = m.step(torch.tensor(CU, dtype=torch.int32).cuda())
    leaves = {n: getattr(m, n).double().requires_grad_() for n in ("x", "w", "b", "a", "norm_w")}
    x = leaves["x"]
    v, mean = torch.var_mean(x, dim=1, keepdim=True, correction=0)
    xn = (x - mean) * torch.rsqrt(v + EPS) * leaves["w"] + leaves["b"]
    u, i, r, z = m.columns(xn @ m.w_in.double().t())
    p = leaves["a"] * torch.sigmoid(r)
    e, b = torch.exp(p), torch.sqrt(-torch.expm1(2 * p)) * torch.sigmoid(i) * u
    rows = []
    for r0, r1 in SPANS:
        h = torch.zeros(WIDTH, dtype=torch.float64, device="cuda")
        for t in range(r0, r1):
            h = e[t] * h + b[t]
            rows.append(h)
    y = (torch.stack(rows) * torch.nn.functional.silu(z)).unflatten(1, (-1, GROUP))
    h = (y * torch.rsqrt((y * y).mean(2, keepdim=True) + EPS)).flatten(1) * leaves["norm_w"]
    want = torch.autograd.grad(h @ m.w_out.double().t(), list(leaves.values()), m.dout.double())
    for n, w, v in zip(leaves, want, (got[12], got[13], got[14], got[10], got[8])):
        # about a dozen roundings of 2^-9 lie between, each of its own sign
        assert (v.double() - w).norm() <= 0.03 * w.norm(), n


def test_a_captured_training_step():
    m = Layer(CU[-1])
    cu = torch.tensor(CU, dtype=torch.int32).cuda()
    m.step(cu)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        got = m.step(cu)
    m.x.copy_(m.x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, m.step(cu)))


COLD = """
import torch, gated_group_rmsnorm_gb300 as g
gen = torch.Generator().manual_seed(0)
x, i, r, z, d = (torch.randn(900, 512, generator=gen).bfloat16().cuda() for _ in range(5))
w, a = torch.randn(512, generator=gen).cuda(), -torch.rand(512, generator=gen).cuda()
torch.cuda.synchronize()

def step():
    y = g.linear_recurrence(x, i, r, a)
    out = (g.layer_norm(x, w, eps=1e-5), y) + g.linear_recurrence_backward(d, x, i, r, a)[:4]
    out += g.layer_norm_backward(d, x, w, eps=1e-5)
    return out + g.backward(d, y, z, w, group_size=64, eps=1e-5)

graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(graph, stream=s):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(u, v) for u, v in zip(got, step()))
assert g.fault_status() == 0
"""


def test_the_first_calls_of_a_process_may_be_captured():
    r = subprocess.run([sys.executable, "-c", COLD], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_two_captured_steps_at_once():
    """Graphs with workspaces of their own, replayed on two streams at the same time."""
    ms, cu = [Layer(CU[-1], seed=k) for k in range(2)], torch.tensor(CU, dtype=torch.int32).cuda()
    want = [m.step(cu) for m in ms]
    graphs, got, streams = [], [], [torch.cuda.Stream() for _ in ms]
    for m in ms:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(m.step(cu))
        graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for a, b in zip(want, got) for u, v in zip(a, b))


def test_calls_from_several_threads():
    ms, cu = [Layer(CU[-1], seed=k) for k in range(3)], torch.tensor(CU, dtype=torch.int32).cuda()
    want = [m.step(cu) for m in ms]
    torch.cuda.synchronize()
    wrong, started = [], threading.Barrier(len(ms))

    def run(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                started.wait(timeout=30)
                for _ in range(20):
                    got = ms[k].step(cu)
                    torch.cuda.current_stream().synchronize()
                    assert all(torch.equal(u, v) for u, v in zip(want[k], got))
        except BaseException as e:  # (an exception of a thread reaches no test by itself)
            wrong.append(e)

    threads = [threading.Thread(target=run, args=(k,)) for k in range(len(ms))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    assert g.fault_status() == 0


def test_decoding_in_a_graph():
    """Layer norm, recurrence step and gated norm replayed: as the same calls made one by
    one; the states advance with each replay."""
    gen = torch.Generator().manual_seed(0)
    batch = 3
    x = torch.randn(batch, MODEL, generator=gen).to(T).cuda()
    proj = torch.randn(batch, 4 * WIDTH, generator=gen).to(T).cuda()
    m = Layer(1)
    u, i, r, z = m.columns(proj)
    slots = torch.tensor([2, 0, 3], dtype=torch.int32).cuda()
    state = torch.randn(4, WIDTH, generator=gen).cuda()
    xn, y, h = (torch.empty(batch, n, dtype=T, device="cuda") for n in (MODEL, WIDTH, WIDTH))
    live = state.clone()
    graph = g.DecodeGraph([
        dict(op="layer_norm", x=x, w=m.w, b=m.b, eps=EPS, out=xn),
        dict(op="linear_recurrence_step", x=u, input_gate=i, decay_gate=r, a=m.a, state=live,
             slots=slots, out=y),
        dict(y=y, gate=z, w=m.norm_w, out=h, group_size=GROUP, eps=EPS)])
    for _ in range(3):
        graph.replay()
        want = (g.layer_norm(x, m.w, m.b, eps=EPS),
                g.linear_recurrence_step(u, i, r, m.a, state, slots=slots))
        want += (g.forward(want[1], z, m.norm_w, group_size=GROUP, eps=EPS),)
        assert all(torch.equal(a, b) for a, b in zip((xn, y, h), want))
        assert torch.equal(live, state)
    # a chain of one call is launched directly
    graph = g.DecodeGraph([dict(op="layer_norm", x=x, w=m.w, eps=EPS, out=xn)])
    graph.replay()
    assert torch.equal(xn, g.layer_norm(x, m.w, eps=EPS))
    with pytest.raises(ValueError, match="takes no gate"):
        g.DecodeGraph([dict(op="layer_norm", x=x, w=m.w, eps=EPS, out=xn, gate=z)])


def test_offsets_past_2_31_elements():
    """Rows 2^30 elements apart: the same bits as from rows beside each other."""
    free, _ = torch.cuda.mem_get_info()
    if free < 40 * 2 ** 30:
        pytest.skip("needs about 30 GB of free device memory")
    rows, width, apart = 4, 512, 1 << 30
    gen = torch.Generator().manual_seed(0)
    near = [torch.randn(rows, width, generator=gen).to(T).cuda() for _ in range(4)]
    whole = torch.zeros(3 * apart + 8 * width, dtype=T, device="cuda")
    far = [torch.as_strided(whole, (rows, width), (apart, 1), k * width) for k in range(8)]
    for f, n in zip(far, near):
        f.copy_(n)
    w = torch.randn(width, generator=gen).cuda()
    a = -torch.rand(width, generator=gen).cuda()
    g.layer_norm(far[0], w, eps=EPS, out=far[4])
    assert torch.equal(far[4], g.layer_norm(near[0], w, eps=EPS))
    got = g.layer_norm_backward(far[0], far[1], w, eps=EPS, dx=far[4])
    want = g.layer_norm_backward(near[0], near[1], w, eps=EPS)
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    got = g.backward(far[0], far[1], far[2], w, group_size=64, eps=EPS, dy=far[4], dgate=far[5])
    want = g.backward(near[0], near[1], near[2], w, group_size=64, eps=EPS)
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    g.linear_recurrence(*far[:3], a, out=far[4])
    assert torch.equal(far[4], g.linear_recurrence(*near[:3], a))
    got = g.linear_recurrence_backward(far[3], *far[:3], a, dx=far[4], dinput_gate=far[5],
                                       ddecay_gate=far[6])
    want = g.linear_recurrence_backward(near[3], *near[:3], a)
    assert all(torch.equal(u, v) for u, v in zip(got[:4], want[:4]))
    st = [torch.zeros(rows, width, device="cuda") for _ in range(2)]
    g.linear_recurrence_step(*far[:3], a, st[0], out=far[4])
    assert torch.equal(far[4], g.linear_recurrence_step(*near[:3], a, st[1]))
    del whole, far
    torch.cuda.empty_cache()


def test_what_the_binding_refuses():
    x = torch.zeros(8, 32, dtype=T, device="cuda")
    v, short = torch.zeros(32, device="cuda"), torch.zeros(31, device="cuda")
    st = torch.zeros(8, 32, device="cuda")
    cu = torch.tensor([0, 8], dtype=torch.int32).cuda()
    bad = [
        lambda: g.linear_recurrence(x, x.float(), x, v),
        lambda: g.linear_recurrence(x, x, x[:4], v),
        lambda: g.linear_recurrence(x, x, x, short),
        lambda: g.linear_recurrence(x, x, x, v.double()),
        lambda: g.linear_recurrence(x, x, x, v, state=st.half()),
        lambda: g.linear_recurrence(x, x, x, v, state=st[:, :16]),
        lambda: g.linear_recurrence(x, x, x, v, slots=cu[:1]),
        lambda: g.linear_recurrence(x, x, x, v, cu_seqlens=cu.long()),
        lambda: g.linear_recurrence(x, x, x, v, saved=torch.zeros(2, 32, device="cuda")),
        lambda: g.linear_recurrence(x, x, x, v, out=torch.zeros(8, 32, device="cuda")),
        lambda: g.linear_recurrence(x.t(), x.t(), x.t(), torch.zeros(8, device="cuda")),
        lambda: g.linear_recurrence_step(x, x, x, v, None),
        lambda: g.linear_recurrence_step(x, x, x, v, st[:4]),
        lambda: g.linear_recurrence_backward(x[:4], x, x, x, v),
        lambda: g.linear_recurrence_backward(x, x, x, x, v, dstate=st),
        lambda: g.linear_recurrence_backward(x, x, x, x, v, saved=st),
        lambda: g.linear_recurrence_backward(x, x, x, x, v, dx=x[:, :16]),
        lambda: g.layer_norm(x, short, eps=EPS),
        lambda: g.layer_norm(x, v.bfloat16(), eps=EPS),
        lambda: g.layer_norm(x.long(), v, eps=EPS),
        lambda: g.layer_norm_backward(x.float(), x, v, eps=EPS),
        lambda: g.layer_norm_backward(x, x, v, eps=EPS, dx=x[:4]),
        lambda: g.backward(x, x, x, short, group_size=8, eps=EPS),
        lambda: g.backward(x, x, x, v, group_size=8, eps=EPS, mode="onnx"),
        lambda: g.backward(x, x, x[:4], v, group_size=8, eps=EPS),
    ]
    for k, call in enumerate(bad):
        with pytest.raises((ValueError, g.GgrnError)):
            call()
            pytest.fail(f"call {k} was taken")
    with pytest.raises(g.GgrnError):   # an output on an input
        g.layer_norm(x, v, eps=EPS, out=x)
    with pytest.raises(g.GgrnError):   # 32 columns are no groups of 5
        g.backward(x, x, x, v, group_size=5, eps=EPS)
