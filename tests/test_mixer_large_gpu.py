"""The mixer's operators at sizes where their launches take more than the
smallest tiles: the convolution's sliding window over several rounds of loads,
four sequences to a thread of its step form, two rounds of rows to a CTA of the
scan's; and the step forms with every option off.  152 SMs are assumed by the
sizes, not by the results."""
import math

import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from tests import mixer_ref as ref
from tests.test_conv_gpu import DTYPES, _close, _inputs
from tests.test_scan_gpu import Case, check_state

pytestmark = pytest.mark.gpu


def _ends(rows, lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    assert cu[-1] <= rows
    return cu


# width, pad, col, rows: tiles of 12, 28, 20 and 64 rows of 16-byte vectors in
# 16-bit types (20, 56, 40 and 64 in f32), of 60 and 24 rows of single channels
CONV = [(2432, 8, 8, 2500), (9728, 0, 0, 2100), (9728, 64, 16, 1531), (4864, 0, 0, 9700),
        (1000, 1, 0, 5600), (3000, 3, 1, 700)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("taps", [2, 4])
@pytest.mark.parametrize("width,pad,col,rows", CONV)
def test_conv_tiles_of_many_rows(dtype, taps, width, pad, col, rows):
    """Ragged sequences that begin and end everywhere in the tiles, one of them
    longer than several, empty ones and one without an entry."""
    lens = [1, 2, 3, 0, 5, 63, 64, 65, 1, 0, rows // 3, 4, 127, 31]
    cu = _ends(rows, lens)
    n = len(lens)
    packed, w, bias, state = _inputs(rows, width, taps, dtype, n, seed=rows, pad=pad, col=col)
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    slots[5] = -1
    resume = torch.tensor([i % 2 == 0 for i in range(n)])
    x = packed.cuda()[:, col:col + width]
    out = torch.full((rows, width), 7.0, dtype=dtype, device="cuda")
    st = state.cuda()
    g.causal_conv(x, w.cuda(), bias.cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(),
                  state=st, slots=slots.cuda(), resume=resume.cuda(), out=out)
    want, bound, new = ref.conv(packed[:, col:col + width], w, bias, spans=ref.ranges(rows, cu),
                                state=state, slots=slots.tolist(), resume=resume.tolist())
    fine = _close(out, want, bound, dtype)
    assert (out.cpu()[~fine] == 7.0).all()
    assert torch.equal(st.cpu(), new)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["silu", None])
def test_conv_of_equal_sequences_in_long_tiles(dtype, act):
    rows, seqs, width = 2058, 7, 4864
    packed, w, bias, state = _inputs(rows, width, 4, dtype, seqs, seed=2)
    x = packed.cuda().view(seqs, rows // seqs, width)
    st = state.cuda()
    got = g.causal_conv(x, w.cuda(), bias.cuda(), activation=act, state=st)
    want, bound, new = ref.conv(packed, w, bias, act is not None, spans=ref.ranges(rows, None, seqs),
                                state=state)
    _close(got.reshape(rows, width), want, bound, dtype)
    assert torch.equal(st.cpu(), new)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("width,pad,act", [(9728, 8, "silu"), (2432, 0, None), (1001, 2, "silu")])
def test_conv_steps_of_many_sequences(dtype, taps, width, pad, act):
    """Batches that are no multiple of four, with rows of padding among them."""
    batch = 1301 if width < 4000 else 331
    packed, w, bias, state = _inputs(batch, width, taps, dtype, batch + 3, pad=pad, seed=taps)
    slots = torch.randperm(batch + 3, generator=torch.Generator().manual_seed(3))[:batch].to(
        torch.int32)
    slots[[0, 5, 6, 7, 9]], slots[batch - 1] = -1, batch + 3
    st = state.cuda()
    out = torch.full((batch, width), 7.0, dtype=dtype, device="cuda")
    g.causal_conv_step(packed.cuda()[:, :width], st, w.cuda(), bias.cuda(), activation=act,
                       slots=slots.cuda(), out=out)
    want, bound, new = ref.conv(packed[:, :width], w, bias, act is not None,
                                spans=[(i, i + 1) for i in range(batch)], state=state,
                                slots=slots.tolist(), step=True)
    fine = _close(out, want, bound, dtype)
    assert (out.cpu()[~fine] == 7.0).all()
    assert torch.equal(st.cpu(), new)


# heads, head_dim, groups, state_size, batch: head_dim full rounds of rows, one
# and a half, and less than one behind a full CTA
SCAN = [(96, 80, 8, 128, 7), (80, 40, 1, 128, 20), (64, 100, 2, 96, 10), (48, 65, 1, 33, 12),
        (30, 64, 3, 256, 25), (70, 130, 1, 12, 40)]


def _step_ok(got, want, bound, dtype):
    """The step forms compute in f32: the f32 bound and the output's rounding."""
    tol = (bound + ref.rounding(want, dtype)) * (1 + 2.0 ** -7)
    fine = ~torch.isnan(want)
    assert ((got.double().cpu() - want).abs() <= tol)[fine].all()
    return fine


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,head_dim,groups,state_size,batch", SCAN)
def test_scan_steps_of_many_sequences(dtype, heads, head_dim, groups, state_size, batch):
    k = Case(batch, heads, head_dim, groups, state_size, dtype, slots=batch + 1, seed=11)
    slots = torch.randperm(batch + 1, generator=torch.Generator().manual_seed(4))[:batch].to(
        torch.int32)
    slots[2] = -1
    st = k.state.cuda()
    out = torch.full((batch, heads * head_dim), 7.0, dtype=dtype, device="cuda")
    v, w = k.on()
    g.ssm_scan_step(v["x"], v["dt"], w["a"], v["b"], v["c"], st, d=w["d"], dt_bias=w["dt_bias"],
                    slots=slots.cuda(), out=out)
    want, bound, size, new, nb, ns = k.want(spans=[(i, i + 1) for i in range(batch)],
                                            slots=slots.tolist(), step=True)
    fine = _step_ok(out, want, bound, dtype)
    assert (out.cpu()[~fine] == 7.0).all()
    check_state(st, new, nb, ns)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("limits,softplus,options", [((0.5, 2.0), True, True),
                                                     ((0.0, math.inf), False, True),
                                                     ((0.25, 0.75), False, False),
                                                     ((0.0, math.inf), True, False)])
def test_scan_steps_with_limits_and_without_options(dtype, limits, softplus, options):
    k = Case(9, 6, 20, 2, 24, dtype, slots=9, seed=12)
    k.z = k.z.abs()
    v, w = k.on()
    st = k.state.cuda()
    kw = dict(d=w["d"], dt_bias=w["dt_bias"]) if options else {}
    got = g.ssm_scan_step(v["x"], v["dt"], w["a"], v["b"], v["c"], st, dt_limits=limits,
                          dt_softplus=softplus, **kw)
    c = k.views(k.xbc, k.z)
    want, bound, size, new, nb, ns = ref.scan(
        c["x"], c["dt"], k.a, c["b"], c["c"], 20, 24, *((k.d, k.dt_bias) if options else ()),
        softplus=softplus, limits=limits, state=k.state, spans=[(i, i + 1) for i in range(9)],
        step=True)
    _step_ok(got, want, bound, dtype)
    check_state(st, new, nb, ns)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("taps", [2, 3, 4])
def test_conv_steps_without_options(dtype, taps):
    packed, w, _, state = _inputs(5, 200, taps, dtype, 5, seed=13)
    st = state.cuda()
    got = g.causal_conv_step(packed.cuda(), st, w.cuda(), activation=None)
    want, bound, new = ref.conv(packed, w, None, False, spans=[(i, i + 1) for i in range(5)],
                                state=state, step=True)
    _close(got, want, bound, dtype)
    assert torch.equal(st.cpu(), new)


# shapes and types of prompts that run token by token in f32, whatever the type
EXACT = [(torch.float16, (4, 64, 1, 128)), (torch.float16, (6, 80, 2, 128)),
         (torch.float16, (2, 5, 1, 3)), (torch.bfloat16, (2, 64, 1, 250)),
         (torch.bfloat16, (2, 130, 1, 256)), (torch.bfloat16, (5, 36, 5, 100)),
         (torch.bfloat16, (2, 5, 1, 16)), (torch.bfloat16, (3, 64, 1, 20))]


@pytest.mark.parametrize("dtype,shape", EXACT)
@pytest.mark.parametrize("decay", [None, -0.0, 0.02])
def test_prompts_token_by_token_round_the_output_only(dtype, shape, decay):
    rows, cu = 400, [2, 3, 40, 40, 397]
    k = Case(rows, *shape, dtype, slots=4, seed=14, dt_shift=0.0 if decay is None else -1.0)
    if decay is not None:
        k.a = torch.full_like(k.a, decay)
    st = k.state.cuda()
    resume = torch.tensor([True, False, True, True])
    out = k.run(cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), state=st,
                resume=resume.cuda())
    want, bound, size, new, nb, ns = k.want(spans=ref.ranges(rows, cu), resume=resume.tolist())
    _step_ok(out, want, bound, dtype)
    check_state(st, new, nb, ns)
