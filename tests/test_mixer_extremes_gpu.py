"""The mixer's operators far out: offsets behind 2^31 elements, many short
sequences, calls at the same time."""
import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from tests import mixer_ref as ref
from tests.test_scan_gpu import Case, check, check_state

pytestmark = pytest.mark.gpu
FAR = 2 ** 31


def _room(nbytes):
    if torch.cuda.mem_get_info()[0] < 2 * nbytes:
        pytest.skip("not enough device memory")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_slots_far_into_the_pools(dtype):
    """The same results from entries whose offsets pass 2^31 elements as from
    the first ones of a small pool, for prompts and single tokens."""
    _room(FAR * 4)
    heads, head_dim, state_size, taps, rows = 16, 64, 128, 4, 150
    k = Case(rows, heads, head_dim, 1, state_size, dtype, slots=2, seed=31)
    v, w = k.on()
    width = v["x"].shape[1]
    cw = torch.randn(width, taps, generator=torch.Generator().manual_seed(5)).cuda()
    cu = torch.tensor([0, 70, rows], dtype=torch.int32).cuda()
    resume = torch.ones(2, dtype=torch.bool).cuda()

    def go(scan_pool, conv_pool, slots):
        kw = dict(d=w["d"], dt_bias=w["dt_bias"], slots=slots)
        outs = [g.causal_conv(v["x"], cw, cu_seqlens=cu, state=conv_pool, slots=slots,
                              resume=resume),
                g.ssm_scan(v["x"], v["dt"], w["a"], v["b"], v["c"], cu_seqlens=cu, resume=resume,
                           state=scan_pool, head_dim=head_dim, state_size=state_size, **kw),
                g.causal_conv_step(v["x"][:2], conv_pool, cw, slots=slots)]
        step = {n: v[n][:2] for n in "x b c dt".split()}
        outs.append(g.ssm_scan_step(step["x"], step["dt"], w["a"], step["b"], step["c"], scan_pool,
                                    **kw))
        at = slots.long()
        return outs + [scan_pool[at], conv_pool[at]]

    first = k.state.cuda()
    conv_first = torch.randn(2, taps - 1, width, generator=torch.Generator().manual_seed(6)).to(
        dtype).cuda()
    entry, conv_entry = first[0].numel(), conv_first[0].numel()
    n = FAR // entry + 2
    m = FAR // conv_entry + 2
    far, conv_far = (torch.empty(n, *first.shape[1:], device="cuda"),
                     torch.empty(m, *conv_first.shape[1:], dtype=dtype, device="cuda"))
    last = min(n, m) - 1  # the smaller entries' pool decides; both pass 2^31 in the other test
    near = go(first.clone(), conv_first.clone(), torch.tensor([1, 0], dtype=torch.int32).cuda())
    far[[n - 1, n - 2]] = first[[1, 0]]
    conv_far[[last, last - 1]] = conv_first[[1, 0]]
    # one index serves both pools: views that end at it
    got = go(far[n - 1 - last:], conv_far, torch.tensor([last, last - 1], dtype=torch.int32).cuda())
    for a, b in zip(near, got):
        assert torch.equal(a, b)
    # the convolution's pool on its own, at its own end
    conv_far[[m - 1, m - 2]] = conv_first[[1, 0]]
    got = g.causal_conv(v["x"], cw, cu_seqlens=cu, state=conv_far, resume=resume,
                        slots=torch.tensor([m - 1, m - 2], dtype=torch.int32).cuda())
    assert torch.equal(got, near[0])
    # and the scan's from its base, the slot's offset itself past 2^31
    far[[n - 1, n - 2]] = first[[1, 0]]
    got = k.run(cu_seqlens=cu, state=far, resume=resume,
                slots=torch.tensor([n - 1, n - 2], dtype=torch.int32).cuda())
    assert torch.equal(got, near[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_far_apart(dtype):
    """Row strides that put the later rows behind 2^31 elements."""
    rows, heads, head_dim, state_size = 520, 4, 32, 64
    stride = FAR // 500 // 64 * 64
    _room(rows * stride * dtype.itemsize)
    k = Case(rows, heads, head_dim, 1, state_size, dtype, seed=33)
    v, w = k.on()
    big = torch.empty(rows, stride, dtype=dtype, device="cuda")
    cuts = k.cuts
    big[:, :cuts[3]] = k.xbc.cuda()
    big[:, cuts[3]:cuts[3] + heads] = v["dt"]
    out = big[:, cuts[3] + 64:cuts[3] + 64 + heads * head_dim]
    kw = dict(head_dim=head_dim, state_size=state_size, d=w["d"], dt_bias=w["dt_bias"])
    near = g.ssm_scan(v["x"], v["dt"], w["a"], v["b"], v["c"], **kw)
    far = k.views(big, big[:, cuts[3] - 3:cuts[3] + heads])
    with pytest.raises(g.GgrnError):  # one buffer's rows interleave: refused
        g.ssm_scan(far["x"], far["dt"], w["a"], far["b"], far["c"], out=out, **kw)
    assert torch.equal(g.ssm_scan(far["x"], far["dt"], w["a"], far["b"], far["c"], **kw), near)
    cw = torch.randn(heads * head_dim, 4, generator=torch.Generator().manual_seed(7)).cuda()
    assert torch.equal(g.causal_conv(far["x"], cw), g.causal_conv(v["x"], cw))
    # far rows of the output
    spread = torch.zeros(rows, stride, dtype=dtype, device="cuda")
    got = spread[:, 64:64 + heads * head_dim]
    g.ssm_scan(v["x"], v["dt"], w["a"], v["b"], v["c"], out=got, **kw)
    assert torch.equal(got, near)
    g.causal_conv(v["x"], cw, out=got)
    assert torch.equal(got, g.causal_conv(v["x"], cw))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_many_short_sequences(dtype):
    gen = torch.Generator().manual_seed(35)
    lens = torch.randint(0, 4, (1500,), generator=gen)
    cu = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)]).to(torch.int32)
    rows = int(cu[-1])
    k = Case(rows, 2, 16, 1, 16, dtype, slots=1500, seed=36)
    st = k.state.cuda()
    out = k.run(cu_seqlens=cu.cuda(), state=st)
    spans = ref.ranges(rows, cu.tolist())
    want, bound, size, new, nb, ns = k.want(spans=spans)
    check(out, want, bound, size, dtype)
    check_state(st, new, nb, ns)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_two_calls_at_once(dtype):
    """On two streams, each with the workspace it takes for itself."""
    cases = [Case(3000, 8, 64, 1, 128, dtype, seed=s) for s in (37, 38)]
    alone = [k.run() for k in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for k, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(k.run())
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert torch.equal(a, b)
    assert g.fault_status() == 0
