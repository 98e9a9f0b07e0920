"""The Python entry of the mixer's operators beside other threads, graphs and
buffers of the caller's."""
import os
import subprocess
import sys
import threading
import time

import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from tests.test_scan_gpu import Case

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_other_threads_run_while_a_call_waits_for_the_launch_queue():
    """A stream kept busy for about half a second, and more calls on it than its
    queue holds: the caller waits, another Python thread does not."""
    k = Case(1, 1, 16, 1, 16, torch.bfloat16, slots=1)
    v, w = k.on()
    st, out = k.state.cuda(), torch.empty(1, 16, dtype=torch.bfloat16, device="cuda")

    def step():
        g.ssm_scan_step(v["x"], v["dt"], w["a"], v["b"], v["c"], st, out=out)

    step()
    torch.cuda.synchronize()
    done = threading.Event()

    def calls():
        torch.cuda._sleep(1_000_000_000)
        for _ in range(6000):
            step()
        done.set()

    worker = threading.Thread(target=calls)
    worst, last = 0.0, time.perf_counter()
    begin = last
    worker.start()
    while not done.is_set():
        time.sleep(0.002)
        now = time.perf_counter()
        worst, last = max(worst, now - last), now
    worker.join()
    whole = time.perf_counter() - begin
    torch.cuda.synchronize()
    assert whole > 0.2, "the queue took every call at once: nothing was tested"
    assert worst < 0.1, (worst, whole)


COLD = """
import torch, gated_group_rmsnorm_gb300 as g
gen = torch.Generator().manual_seed(0)
heads, P, N, rows = 4, 64, 128, 2500
x, b, c = (torch.randn(rows, n, generator=gen).bfloat16().cuda() for n in (heads * P, N, N))
dt = torch.randn(rows, heads, generator=gen).bfloat16().cuda()
a = -torch.rand(heads, generator=gen).cuda()
w = torch.randn(heads * P, 4, generator=gen).cuda()
torch.cuda.synchronize()
graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(graph, stream=s):
    u = g.causal_conv(x, w)
    y = g.ssm_scan(u, dt, a, b, c, head_dim=P, state_size=N)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(u, g.causal_conv(x, w))
assert torch.equal(y, g.ssm_scan(u, dt, a, b, c, head_dim=P, state_size=N))
assert g.fault_status() == 0
"""


def test_the_first_call_of_a_process_may_be_captured():
    r = subprocess.run([sys.executable, "-c", COLD], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_calls_from_several_threads(dtype):
    """Calls of several threads at the same time, each on a stream of its own."""
    cases = [Case(900 + 100 * i, 4, 64, 1, 96, dtype, seed=20 + i) for i in range(4)]
    w = torch.randn(256, 4, generator=torch.Generator().manual_seed(1)).cuda()
    inputs = [k.on() for k in cases]

    def both(v, c):
        return (g.causal_conv(v["x"], w),
                g.ssm_scan(v["x"], v["dt"], c["a"], v["b"], v["c"], head_dim=64, state_size=96,
                           d=c["d"], dt_bias=c["dt_bias"]))

    want = [both(*i) for i in inputs]
    torch.cuda.synchronize()
    wrong, started = [], threading.Barrier(len(cases))

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                started.wait(timeout=30)
                for _ in range(40):
                    got = both(*inputs[i])
                    torch.cuda.current_stream().synchronize()
                    assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
        except BaseException as e:  # (an exception of a thread reaches no test by itself)
            wrong.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    assert g.fault_status() == 0
