"""The causal convolution on the GPU against its definition in 64 bits."""
import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from tests import mixer_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _inputs(rows, width, taps, dtype, slots, seed=0, pad=0, col=0):
    gen = torch.Generator().manual_seed(seed)
    packed = torch.randn(rows, col + width + pad, generator=gen).to(dtype)
    w = torch.randn(width, taps, generator=gen)
    bias = torch.randn(width, generator=gen)
    state = torch.randn(slots, taps - 1, width, generator=gen).to(dtype)
    return packed, w, bias, state


def _close(got, want, bound, dtype):
    got = got.double().cpu()
    tol = bound + ref.rounding(want, dtype) * (1 + 2.0 ** -8)
    fine = ~torch.isnan(want)
    worst = ((got - want).abs() - tol)[fine]
    assert worst.numel() == 0 or worst.max() <= 0, worst.max()
    return fine


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("width,pad,col", [(64, 0, 0), (1064, 16, 8), (37, 3, 1), (8, 1, 0)])
def test_ragged_prompts(dtype, taps, width, pad, col):
    """Sequences of 0, 1, 2, 3, ... rows and long ones, some resumed, one
    without an entry, rows in front of the first and behind the last."""
    cu = [2, 2, 3, 5, 8, 8, 12, 50, 83]
    rows, n = 90, len(cu) - 1
    packed, w, bias, state = _inputs(rows, width, taps, dtype, n + 2, pad=pad, col=col)
    slots = torch.tensor([4, 9, 0, 7, 2, 3, -1, 1], dtype=torch.int32)  # pool of 10
    resume = torch.tensor([1, 0, 1, 1, 0, 1, 1, 0], dtype=torch.bool)
    dev = packed.cuda()
    x = dev[:, col:col + width]
    out = torch.full((rows, width), 7.0, dtype=dtype, device="cuda")
    st = state.cuda()
    g.causal_conv(x, w.cuda(), bias.cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(),
                  state=st, slots=slots.cuda(), resume=resume.cuda(), out=out)
    want, bound, new = ref.conv(packed[:, col:col + width], w, bias, spans=ref.ranges(rows, cu),
                                state=state, slots=slots.tolist(), resume=resume.tolist())
    fine = _close(out, want, bound, dtype)
    assert (out.cpu()[~fine] == 7.0).all()        # rows of no sequence
    assert torch.equal(st.cpu(), new)             # the last inputs, bit for bit


@pytest.mark.parametrize("dtype", DTYPES)
def test_batch_without_offsets_bias_or_state(dtype):
    packed, w, _, _ = _inputs(3 * 21, 48, 4, dtype, 1)
    x = packed.cuda().view(3, 21, 48)
    got = g.causal_conv(x, w.cuda(), activation=None)
    want, bound, _ = ref.conv(packed, w, None, False, spans=ref.ranges(63, None, 3))
    assert got.shape == x.shape
    _close(got.reshape(63, 48), want, bound, dtype)


@pytest.mark.parametrize("rows", [1, 15, 16, 17, 1000])
def test_one_sequence_tile_edges(rows):
    packed, w, bias, state = _inputs(rows, 264, 4, torch.bfloat16, 1, seed=rows)
    st = state.cuda()
    got = g.causal_conv(packed.cuda(), w.cuda(), bias.cuda(), state=st)
    want, bound, new = ref.conv(packed, w, bias, spans=[(0, rows)], state=state)
    _close(got, want, bound, torch.bfloat16)
    assert torch.equal(st.cpu(), new)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("width,pad", [(1288, 8), (21, 0)])
def test_steps(dtype, taps, width, pad):
    batch = 5
    packed, w, bias, state = _inputs(batch, width, taps, dtype, 7, pad=pad)
    slots = torch.tensor([6, 0, -1, 3, 7], dtype=torch.int32)  # two rows of padding
    st = state.cuda()
    x = packed.cuda()[:, :width]
    out = torch.full((batch, width), 7.0, dtype=dtype, device="cuda")
    g.causal_conv_step(x, st, w.cuda(), bias.cuda(), slots=slots.cuda(), out=out)
    want, bound, new = ref.conv(packed[:, :width], w, bias, spans=[(i, i + 1) for i in range(batch)],
                                state=state, slots=slots.tolist(), step=True)
    fine = _close(out, want, bound, dtype)
    assert (out.cpu()[~fine] == 7.0).all()
    assert torch.equal(st.cpu(), new)


def test_prompt_then_steps_is_the_whole_prompt():
    """Cut anywhere, the convolution gives the same bits."""
    rows, width = 23, 96
    packed, w, bias, _ = _inputs(rows, width, 4, torch.float16, 1)
    x, w, bias = packed.cuda(), w.cuda(), bias.cuda()
    whole = g.causal_conv(x, w, bias)
    for cut in (0, 1, 2, 3, 4, 20):
        st = torch.full((1, 3, width), 9.0, dtype=torch.float16, device="cuda")
        parts = []
        fresh = torch.zeros(1, dtype=torch.bool, device="cuda")
        if cut:
            parts.append(g.causal_conv(x[:cut], w, bias, state=st, resume=fresh))
        else:  # an empty prompt leaves zeros
            g.causal_conv(x[:0], w, bias, state=st,
                          cu_seqlens=torch.zeros(2, dtype=torch.int32, device="cuda"))
        for t in range(cut, rows):
            parts.append(g.causal_conv_step(x[t:t + 1], st, w, bias))
        assert torch.equal(torch.cat(parts), whole)


def test_nan_and_inf_stay_in_their_window():
    rows, width = 40, 16
    packed, w, bias, _ = _inputs(rows, width, 4, torch.bfloat16, 1)
    packed[10, 3], packed[30, 5] = float("nan"), float("inf")
    cu = torch.tensor([0, 12, 40], dtype=torch.int32).cuda()
    got = g.causal_conv(packed.cuda(), w.cuda(), bias.cuda(), cu_seqlens=cu, activation=None).cpu()
    odd = ~torch.isfinite(got)
    assert odd[10:12, 3].all() and odd[30:34, 5].all() and int(odd.sum()) == 6


def test_offsets_out_of_range_are_clamped():
    """Offsets outside the rows lead nowhere outside the buffers."""
    rows, width = 20, 32
    packed, w, bias, state = _inputs(rows, width, 4, torch.float32, 3)
    guard = torch.full((rows + 8, width), 7.0, device="cuda")
    st = state.cuda()
    cu = torch.tensor([-5, 6, 1000000, 7], dtype=torch.int32).cuda()
    g.causal_conv(packed.cuda(), w.cuda(), bias.cuda(), cu_seqlens=cu, state=st,
                  out=guard[:rows])
    assert (guard[rows:] == 7.0).all()
    want, bound, _ = ref.conv(packed, w, bias, spans=[(0, 6)])
    _close(guard[:6], want[:6], bound[:6], torch.float32)


def test_captured_and_on_another_stream():
    rows, width = 33, 128
    packed, w, bias, state = _inputs(rows, width, 4, torch.bfloat16, 2)
    x, w, bias = packed.cuda(), w.cuda(), bias.cuda()
    st = state.cuda()
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        want = g.causal_conv(x, w, bias).clone()
        g.causal_conv(x, w, bias, state=st, out=out)
        with torch.cuda.graph(graph, stream=side):
            g.causal_conv(x, w, bias, state=st, out=out)
    x.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, g.causal_conv(x, w, bias)) and not torch.equal(out, want)
    assert torch.equal(st[0], x[-3:])
