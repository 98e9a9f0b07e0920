"""The gated linear recurrence and its backward pass on the GPU against their
definitions in 64 bits."""
import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from tests import train_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
RAGGED = [2, 2, 3, 5, 8, 8, 12, 50, 83, 83, 300]  # rows in front of the first sequence, empty ones
SLOTS = [4, 11, 0, 7, 2, 3, -1, 1, 5, 6]          # pool of 12; one sequence has no entry
RESUME = [1, 0, 1, 1, 0, 1, 1, 0, 0, 1]


class Case:
    """Inputs on the host: x and both gates are columns of one projection."""

    def __init__(self, rows, width, dtype, seqs=0, seed=0, pad=0, col=0, rate=0.1):
        gen = torch.Generator().manual_seed(seed)
        self.rows, self.width, self.dtype, self.col = rows, width, dtype, col
        self.proj = torch.randn(rows, col + 3 * width + pad, generator=gen).to(dtype)
        self.a = -rate * torch.rand(width, generator=gen)
        self.state = torch.randn(max(seqs, 1), width, generator=gen)
        self.dout = torch.randn(rows, width, generator=gen).to(dtype)
        self.dstate = torch.randn(max(seqs, 1), width, generator=gen)

    def views(self, proj):
        return [proj[:, self.col + k * self.width:self.col + (k + 1) * self.width]
                for k in range(3)]

    def host(self):
        return self.views(self.proj)

    def cuda(self):
        return self.views(self.proj.cuda())


def _ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _check(case, spans, cu=None, state=None, slots=None, resume=None, batch=None):
    """Forward with kept states, then backward with and without them."""
    x, i, r = case.cuda()
    a = case.a.cuda()
    if batch:
        x, i, r = (t.unflatten(0, (batch, -1)) for t in (x, i, r))
    kw = dict(cu_seqlens=None if cu is None else _ints(cu))
    if state is not None:
        kw.update(slots=None if slots is None else _ints(slots),
                  resume=None if resume is None else torch.tensor(resume, dtype=torch.bool).cuda())
    pool = None if state is None else state.cuda()
    out = torch.full_like(x, 7.0, memory_format=torch.contiguous_format)
    saved = g.linear_recurrence_saved(x)
    saved.fill_(float("nan"))
    g.linear_recurrence(x, i, r, a, state=pool, saved=saved, out=out, **kw)
    want, bound, new, new_bound, before, before_bound = ref.recur(
        *case.host(), case.a, spans, state, slots, resume)
    flat = out.reshape(case.rows, case.width)
    fine = ref.assert_close(flat, want, bound, case.dtype, "out")
    assert (flat.cpu()[~fine] == 7.0).all()
    if state is not None:
        ref.assert_close(pool, new, new_bound, torch.float32, "state")
    at = [t for q in spans for t in range(*q) if t % 64 == 0 and t != q[0]]
    ref.assert_close(saved.cpu()[[t // 64 for t in at]], before[at], before_bound[at],
                     torch.float32, "saved")

    dout = case.dout.cuda().reshape(x.shape)
    dstate = case.dstate[:len(spans)].cuda()
    old = None if state is None else state.cuda()
    grads = ref.recur_backward(case.dout, *case.host(), case.a, spans, state, slots, resume,
                               case.dstate)
    first = None
    for kept in (saved, None):
        got = g.linear_recurrence_backward(dout, x, i, r, a, state=old, dstate=dstate, saved=kept,
                                           **kw)
        for n, v in zip(("dx", "di", "dr", "da", "dh"), got):
            if n == "dh" and state is None:
                assert v is None
                continue
            w, b = grads[n]
            ref.assert_close(v.reshape(w.shape), w, b,
                             case.dtype if n in ("dx", "di", "dr") else torch.float32, n)
        assert all((v.reshape(case.rows, case.width).cpu()[~fine] == 0).all() for v in got[:3])
        if first is None:
            first = got
        else:  # the states made again are those that were kept
            assert all(torch.equal(u, v) for u, v in zip(first, got) if u is not None)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width,pad,col,rate", [(64, 0, 0, 0.1), (200, 16, 8, 3.0), (37, 3, 1, 0.1),
                                                (130, 1, 0, 40.0), (1, 0, 0, 1.0)])
def test_ragged_sequences(dtype, width, pad, col, rate):
    """Sequences of 0, 1, 2, 3, .. rows and long ones, some resumed, one without an
    entry, rows in front of the first and behind the last."""
    case = Case(307, width, dtype, 12, pad=pad, col=col, rate=rate)
    _check(case, ref.ranges(307, RAGGED), RAGGED, case.state, SLOTS, RESUME)


@pytest.mark.parametrize("rows", [1, 2, 63, 64, 65, 128, 513, 1100])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_sequence(rows, dtype):
    """Tiles, clusters and their turns at their edges; slow channels beside fast ones."""
    case = Case(rows, 70, dtype, 1, seed=rows, rate=0.3)
    case.a[:35] *= 0.01
    _check(case, [(0, rows)], None, case.state, None, [1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("batch,length", [(3, 21), (5, 64), (4, 200), (9, 130)])
def test_batch_without_offsets_or_state(dtype, batch, length):
    case = Case(batch * length, 48, dtype, batch)
    _check(case, ref.ranges(batch * length, None, batch), batch=batch)


def test_more_clusters_than_one_turn_holds():
    """One long sequence of few channels, and many channels of few rows."""
    case = Case(2500, 6, torch.bfloat16, 1, seed=1, rate=0.01)
    _check(case, [(0, 2500)], None, case.state, None, [1])
    case = Case(70, 11000, torch.bfloat16, 1, seed=2)
    _check(case, [(0, 70)])


def test_segments_of_packed_sequences():
    """Sequences enough that the rows are shared out at their starts."""
    gen = torch.Generator().manual_seed(5)
    cu = [0] + sorted(torch.randint(0, 4000, (29,), generator=gen).tolist()) + [4000]
    case = Case(4003, 34, torch.float16, 30, seed=7)
    _check(case, ref.ranges(4003, cu), cu, case.state, list(range(29, -1, -1)), [1, 0, 1] * 10)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width,pad", [(1288, 8), (21, 0), (6, 1)])
def test_steps(dtype, width, pad):
    case = Case(5, width, dtype, 7, pad=pad, rate=2.0)
    slots = [6, 0, -1, 3, 7]  # two rows of padding
    x, i, r = case.cuda()
    pool, out = case.state.cuda(), torch.full((5, width), 7.0, dtype=dtype, device="cuda")
    g.linear_recurrence_step(x, i, r, case.a.cuda(), pool, slots=_ints(slots), out=out)
    want, bound, new, new_bound, _, _ = ref.recur(*case.host(), case.a,
                                                  [(k, k + 1) for k in range(5)], case.state,
                                                  slots, step=True)
    fine = ref.assert_close(out, want, bound, dtype)
    assert (out.cpu()[~fine] == 7.0).all()
    ref.assert_close(pool, new, new_bound, torch.float32)


def test_prompt_then_steps_is_near_the_whole_prompt():
    rows, width = 150, 96
    case = Case(rows, width, torch.float32, 1, rate=0.05)
    x, i, r = case.cuda()
    a = case.a.cuda()
    want, bound, *_ = ref.recur(*case.host(), case.a, [(0, rows)])
    for cut in (1, 64, 149):
        st = torch.full((1, width), 9.0, device="cuda")
        parts = [g.linear_recurrence(x[:cut], i[:cut], r[:cut], a, state=st)]
        parts += [g.linear_recurrence_step(x[t:t + 1], i[t:t + 1], r[t:t + 1], a, st)
                  for t in range(cut, rows)]
        ref.assert_close(torch.cat(parts), want, bound, torch.float32, cut)


def test_closed_gates_and_decays_of_one():
    """Logits far out on both sides and a = 0: no gradient is a NaN."""
    rows, width = 70, 64
    case = Case(rows, width, torch.float32, 1)
    case.proj[:, width:2 * width][::3] = -80.0
    case.proj[:, 2 * width:][1::3] = -80.0
    case.proj[:, 2 * width:][2::5] = 80.0
    case.a[:4] = 0.0
    _check(case, [(0, rows)])


def test_nan_and_inf_stay_in_their_sequence_and_channel():
    rows, width = 200, 80
    case = Case(rows, width, torch.bfloat16, 3)
    x = case.proj[:, :width]
    x[10, 3], x[130, 5] = float("nan"), float("inf")
    cu = [0, 70, 150, 200]
    x, i, r = case.cuda()
    got = g.linear_recurrence(x, i, r, case.a.cuda(), cu_seqlens=_ints(cu)).cpu()
    odd = ~torch.isfinite(got)
    assert odd[10:70, 3].all() and odd[130:150, 5].all() and int(odd.sum()) == 60 + 20
    dout = case.dout.cuda()
    dout[100, 7] = float("nan")
    dx, *_ = g.linear_recurrence_backward(dout, x, i, r, case.a.cuda(), cu_seqlens=_ints(cu))
    odd = torch.isnan(dx.cpu())
    assert odd[70:101, 7].all() and int(odd[:, 7].sum()) == 31 and not odd[:, :3].any()


def test_offsets_out_of_range_are_clamped():
    rows, width = 100, 32
    case = Case(rows, width, torch.float32, 3)
    guard = [torch.full((rows + 8, width), 7.0, device="cuda") for _ in range(4)]
    x, i, r = case.cuda()
    cu = _ints([-5, 6, 1000000, 7])
    st = case.state.cuda()
    g.linear_recurrence(x, i, r, case.a.cuda(), cu_seqlens=cu, state=st, out=guard[0][:rows])
    g.linear_recurrence_backward(case.dout.cuda(), x, i, r, case.a.cuda(), cu_seqlens=cu,
                                 dx=guard[1][:rows], dinput_gate=guard[2][:rows],
                                 ddecay_gate=guard[3][:rows])
    assert all((t[rows:] == 7.0).all() for t in guard)
    want, bound, *_ = ref.recur(*case.host(), case.a, [(0, 6)])
    ref.assert_close(guard[0][:6], want[:6], bound[:6], torch.float32)


def test_gradients_into_columns_of_one_tensor():
    rows, width = 90, 50
    case = Case(rows, width, torch.bfloat16, 1)
    x, i, r = case.cuda()
    whole = torch.full((rows, 3 * width + 2), 7.0, dtype=torch.bfloat16, device="cuda")
    dx, di, dr = (whole[:, k * width:(k + 1) * width] for k in range(3))
    want = g.linear_recurrence_backward(case.dout.cuda(), x, i, r, case.a.cuda())
    got = g.linear_recurrence_backward(case.dout.cuda(), x, i, r, case.a.cuda(), dx=dx,
                                       dinput_gate=di, ddecay_gate=dr)
    assert got[0].data_ptr() == dx.data_ptr() and (whole[:, 3 * width:] == 7.0).all()
    assert all(torch.equal(u, v) for u, v in zip(want[:4], got[:4]))


def test_no_rows():
    """Empty calls leave states as they are or zero, and give gradients of zero."""
    width = 40
    none = torch.zeros(0, width, device="cuda")
    a = -torch.rand(width).cuda()
    st = torch.ones(3, width, device="cuda")
    cu, resume = _ints([0, 0, 0]), torch.tensor([True, False]).cuda()
    g.linear_recurrence(none, none, none, a, cu_seqlens=cu, state=st, resume=resume,
                        slots=_ints([2, 0]))
    assert (st[2] == 1).all() and (st[0] == 0).all() and (st[1] == 1).all()
    dstate = torch.randn(2, width, device="cuda")
    dx, di, dr, da, dh = g.linear_recurrence_backward(none, none, none, none, a, cu_seqlens=cu,
                                                      state=st, resume=resume, slots=_ints([2, 0]),
                                                      dstate=dstate)
    assert dx.shape == (0, width) and (da == 0).all()
    assert torch.equal(dh[0], dstate[0]) and (dh[1] == 0).all()


def test_captured_and_on_another_stream():
    rows, width = 400, 128
    case = Case(rows, width, torch.bfloat16, 2)
    x, i, r = case.cuda()
    a, dout, st = case.a.cuda(), case.dout.cuda(), case.state.cuda()
    resume = torch.ones(1, dtype=torch.bool, device="cuda")
    out, saved = torch.empty_like(x), g.linear_recurrence_saved(x)

    def both():
        g.linear_recurrence(x, i, r, a, state=st, resume=resume, saved=saved, out=out)
        return (out,) + g.linear_recurrence_backward(dout, x, i, r, a)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
        with torch.cuda.graph(graph, stream=side):
            got = both()
    x.copy_(x.flip(0))
    st.copy_(case.state)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in got if t is not None]
    st.copy_(case.state)
    want = [t for t in both() if t is not None]
    assert all(torch.equal(u, v) for u, v in zip(want, got))


def test_the_same_bits_every_time():
    case = Case(3000, 700, torch.bfloat16, 1, rate=0.02)
    x, i, r = case.cuda()
    a, dout = case.a.cuda(), case.dout.cuda()
    first = None
    for _ in range(5):
        got = (g.linear_recurrence(x, i, r, a),) + g.linear_recurrence_backward(dout, x, i, r, a)[:4]
        first = first or got
        assert all(torch.equal(u, v) for u, v in zip(first, got))


def test_many_sequences_most_of_them_empty():
    """66000 sequences of 300 rows: their states, and the gradients of those."""
    n, rows, width = 66000, 300, 40
    gen = torch.Generator().manual_seed(0)
    cu = torch.sort(torch.randint(0, rows + 1, (n + 1,), generator=gen)).values.to(torch.int32)
    cu[0], cu[-1] = 0, rows
    case = Case(rows, width, torch.float32, 1)
    state = torch.randn(n, width, generator=gen)
    resume = torch.arange(n) % 2 == 0
    spans = [(int(cu[k]), int(cu[k + 1])) for k in range(n)]
    some = [k for k in range(n) if spans[k][1] > spans[k][0]]
    x, i, r = case.cuda()
    st = state.cuda()
    out = g.linear_recurrence(x, i, r, case.a.cuda(), cu_seqlens=cu.cuda(), state=st,
                              resume=resume.cuda())
    # (the same without the empty ones)
    want, bound, new, new_bound, *_ = ref.recur(*case.host(), case.a, [spans[k] for k in some],
                                                state[some], None, resume[some].tolist())
    ref.assert_close(out, want, bound, torch.float32)
    ref.assert_close(st[some], new, new_bound, torch.float32)
    empty = torch.ones(n, dtype=torch.bool)
    empty[some] = False
    assert torch.equal(st.cpu()[empty], state[empty] * resume[empty, None])
    dstate = torch.randn(n, width, generator=gen)
    got = g.linear_recurrence_backward(case.dout.cuda(), x, i, r, case.a.cuda(),
                                       cu_seqlens=cu.cuda(), state=state.cuda(),
                                       resume=resume.cuda(), dstate=dstate.cuda())
    grads = ref.recur_backward(case.dout, *case.host(), case.a, [spans[k] for k in some],
                               state[some], None, resume[some].tolist(), dstate[some])
    for name, v in zip(("dx", "di", "dr", "da"), got):
        ref.assert_close(v, *grads[name], torch.float32, name)
    ref.assert_close(got[4][some], *grads["dh"], torch.float32, "dh")
    assert torch.equal(got[4].cpu()[empty], dstate[empty] * resume[empty, None])
