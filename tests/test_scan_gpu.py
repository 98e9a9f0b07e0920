"""The state space scan on the GPU against its definition in 64 bits."""
import math

import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from tests import mixer_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


class Case:
    """Inputs of one scan on the CPU; `on()` copies them to the GPU with their
    layout (x, b, c columns of one buffer, dt columns of another)."""

    def __init__(self, rows, heads, head_dim, groups, state_size, dtype, slots=0, seed=0, col=0,
                 dt_shift=0.0):
        gen = torch.Generator().manual_seed(seed)
        self.rows, self.heads, self.groups, self.dtype = rows, heads, groups, dtype
        self.head_dim, self.state_size, self.col = head_dim, state_size, col
        inner, gn = heads * head_dim, groups * state_size
        self.cuts = (col, col + inner, col + inner + gn, col + inner + 2 * gn)
        v = torch.randn(rows, self.cuts[3], generator=gen)
        self.xbc = torch.nn.functional.silu(v).to(dtype)
        self.z = torch.randn(rows, 3 + heads, generator=gen).to(dtype)
        dt0 = torch.exp(torch.rand(heads, generator=gen) * math.log(100) + math.log(0.001))
        self.dt_bias = dt0 + torch.log(-torch.expm1(-dt0)) + dt_shift
        self.a = -(1 + 15 * torch.rand(heads, generator=gen))
        self.d = torch.randn(heads, generator=gen)
        self.state = torch.randn(max(slots, 1), heads, head_dim, state_size, generator=gen)
        if not slots:
            self.state = None

    def views(self, xbc, z):
        c0, c1, c2, c3 = self.cuts
        return dict(x=xbc[:, c0:c1], b=xbc[:, c1:c2], c=xbc[:, c2:c3], dt=z[:, 3:])

    def on(self):
        v = self.views(self.xbc.cuda(), self.z.cuda())
        return v, dict(a=self.a.cuda(), d=self.d.cuda(), dt_bias=self.dt_bias.cuda())

    def want(self, **kw):
        v = self.views(self.xbc, self.z)
        if self.state is not None:
            kw.setdefault("state", self.state)
        return ref.scan(v["x"], v["dt"], self.a, v["b"], v["c"], self.head_dim, self.state_size,
                        self.d, self.dt_bias, **kw)

    def run(self, **kw):
        v, w = self.on()
        return g.ssm_scan(v["x"], v["dt"], w["a"], v["b"], v["c"], head_dim=self.head_dim,
                          state_size=self.state_size, d=w["d"], dt_bias=w["dt_bias"], **kw)


def check(got, want, bound, size, dtype):
    """Within the f32 bound, the output's own rounding and, for the types that
    go through the tensor cores, one rounding of an operand to that type
    (relative to the sum of the terms' sizes).  Returns the rows of sequences."""
    got = got.double().cpu()
    fine = ~torch.isnan(want)
    tol = (bound + ref.rounding(want, dtype)) * (1 + 2.0 ** -7)
    if dtype != torch.float32:
        tol = tol + size * (torch.finfo(dtype).eps / 2) * (1 + 2.0 ** -6)
    worst = ((got - want).abs() / tol)[fine]
    assert worst.numel() == 0 or worst.max() <= 1, worst.max()
    return fine


def check_state(got, want, bound, size):
    """f32 states; the tensor cores' operands carry three pieces of 8 bits, so
    a term is off by 2^-24 as in f32: four more of those for their sum."""
    tol = bound + 8 * ref.U * size
    worst = ((got.double().cpu() - want).abs() / (tol + 1e-40))
    assert worst.max() <= 1, worst.max()


SHAPES = [  # heads, head_dim, groups, state_size
    (4, 64, 1, 128), (6, 80, 2, 128), (3, 128, 3, 64), (4, 100, 1, 16), (2, 5, 1, 3),
    (1, 1, 1, 1), (2, 130, 1, 256), (5, 36, 5, 100), (8, 64, 2, 96), (3, 88, 1, 40),
    (1, 1030, 1, 12), (2, 256, 1, 250),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_ragged_prompts(dtype, shape):
    cu = [2, 2, 3, 8, 135, 135, 210]
    rows, n = 220, len(cu) - 1
    k = Case(rows, *shape, dtype, slots=n + 2, col=8)
    slots = torch.tensor([4, 7, 0, 3, 2, 1], dtype=torch.int32)
    resume = torch.tensor([1, 0, 1, 1, 0, 1], dtype=torch.bool)
    out = torch.full((rows, shape[0] * shape[1]), 7.0, dtype=dtype, device="cuda")
    st = k.state.cuda()
    k.run(cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), state=st, slots=slots.cuda(),
          resume=resume.cuda(), out=out)
    want, bound, size, new, nb, ns = k.want(spans=ref.ranges(rows, cu), slots=slots.tolist(),
                                            resume=resume.tolist())
    fine = check(out, want, bound, size, dtype)
    assert (out.cpu()[~fine] == 7.0).all()
    check_state(st, new, nb, ns)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,seqs", [(1, 1), (7, 7), (128, 1), (129, 1), (2 * 257, 2)])
def test_equal_sequences_without_offsets(dtype, rows, seqs):
    k = Case(rows, 4, 64, 2, 128, dtype, slots=seqs, seed=rows)
    st = k.state.cuda()
    got = k.run(state=st) if seqs == 1 else None
    if got is None:
        v, w = k.on()
        three = {n: t.unflatten(0, (seqs, rows // seqs)) for n, t in v.items()}
        got = g.ssm_scan(three["x"], three["dt"], w["a"], three["b"], three["c"], head_dim=64,
                         state_size=128, d=w["d"], dt_bias=w["dt_bias"], state=st)
        got = got.flatten(0, 1)
    want, bound, size, new, nb, ns = k.want(spans=ref.ranges(rows, None, seqs))
    check(got, want, bound, size, dtype)
    check_state(st, new, nb, ns)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1, 64, 1, 128), (2, 80, 1, 128), (1, 24, 1, 16)])
def test_a_long_sequence_is_cut(dtype, shape):
    """Long enough for many parts; beside it short ones and an empty one."""
    cu = [0, 5, 2005, 2005, 2105]
    k = Case(2110, *shape, dtype, slots=4, seed=3)
    args = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    v, w = k.on()
    assert g.scan_workspace_bytes(v["x"], v["dt"], w["a"], v["b"], v["c"], head_dim=shape[1],
                                  state_size=shape[3], **args) > 0
    st = k.state.cuda()
    resume = torch.tensor([0, 1, 1, 0], dtype=torch.uint8)
    out = torch.full((2110, shape[0] * shape[1]), 7.0, dtype=dtype, device="cuda")
    k.run(state=st, resume=resume.cuda(), out=out, **args)
    want, bound, size, new, nb, ns = k.want(spans=ref.ranges(2110, cu), resume=resume.tolist())
    fine = check(out, want, bound, size, dtype)
    assert (out.cpu()[~fine] == 7.0).all()
    check_state(st, new, nb, ns)


@pytest.mark.parametrize("dtype,heads", [(torch.bfloat16, 160), (torch.float32, 500)])
def test_a_long_sequence_in_one_part(dtype, heads):
    """Enough heads to fill the GPU: many chunks one after the other."""
    rows = 1200 if heads == 160 else 200
    k = Case(rows, heads, 16, 1, 40, dtype, slots=1, seed=9)
    v, w = k.on()
    assert g.scan_workspace_bytes(v["x"], v["dt"], w["a"], v["b"], v["c"], head_dim=16,
                                  state_size=40) == 0
    st = k.state.cuda()
    got = k.run(state=st, resume=torch.ones(1, dtype=torch.bool).cuda())
    want, bound, size, new, nb, ns = k.want(spans=[(0, rows)], resume=[True])
    check(got, want, bound, size, dtype)
    check_state(st, new, nb, ns)
    assert g.fault_status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("a,dt_shift,limits", [
    (-0.0, 0.0, (0.0, math.inf)),       # no decay: long sums
    (-16.0, 9.0, (0.0, math.inf)),      # decays that underflow within a token or two
    (-1.0, 3.0, (0.5, 2.0)),            # clamped on both sides
    (0.02, -1.0, (0.0, math.inf)),      # growth
    (-400.0, 2.0, (0.0, math.inf)),     # the exponent far out of range
])
def test_decays(dtype, a, dt_shift, limits):
    k = Case(300, 4, 64, 2, 64, dtype, slots=1, dt_shift=dt_shift)
    k.a = torch.full_like(k.a, a)
    st = k.state.cuda()
    resume = torch.ones(1, dtype=torch.bool).cuda()
    got = k.run(state=st, resume=resume, dt_limits=limits)
    want, bound, size, new, nb, ns = k.want(spans=[(0, 300)], resume=[True], limits=limits)
    check(got, want, bound, size, dtype)
    check_state(st, new, nb, ns)


@pytest.mark.parametrize("dtype", DTYPES)
def test_plain_dt_without_options(dtype):
    k = Case(70, 2, 64, 1, 64, dtype)
    k.z = k.z.abs()
    v, w = k.on()
    got = g.ssm_scan(v["x"], v["dt"], w["a"], v["b"], v["c"], head_dim=64, state_size=64,
                     dt_softplus=False)
    c = k.views(k.xbc, k.z)
    want, bound, size, *_ = ref.scan(c["x"], c["dt"], k.a, c["b"], c["c"], 64, 64, softplus=False,
                                     spans=[(0, 70)])
    check(got, want, bound, size, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_steps(dtype, shape):
    batch = 5
    k = Case(batch, *shape, dtype, slots=7)
    slots = torch.tensor([6, 0, -1, 3, 7], dtype=torch.int32)
    st = k.state.cuda()
    out = torch.full((batch, shape[0] * shape[1]), 7.0, dtype=dtype, device="cuda")
    v, w = k.on()
    g.ssm_scan_step(v["x"], v["dt"], w["a"], v["b"], v["c"], st, d=w["d"], dt_bias=w["dt_bias"],
                    slots=slots.cuda(), out=out)
    want, bound, size, new, nb, ns = k.want(spans=[(i, i + 1) for i in range(batch)],
                                            slots=slots.tolist(), step=True)
    fine = ~torch.isnan(want)
    got = out.double().cpu()
    tol = (bound + ref.rounding(want, dtype)) * (1 + 2.0 ** -7)
    assert ((got - want).abs() <= tol)[fine].all()
    assert (out.cpu()[~fine] == 7.0).all()
    check_state(st, new, nb, ns)
    untouched = [1, 2, 4, 5]
    assert torch.equal(st.cpu()[untouched], k.state[untouched])


def test_entries_inside_a_larger_cache():
    """Pool entries that lie apart, in a cache that holds more than states."""
    k = Case(9, 2, 16, 1, 12, torch.float32, slots=3)
    cache = torch.full((3, 500), 7.0, device="cuda")
    st = cache[:, 4:4 + 2 * 16 * 12].view(3, 2, 16, 12)
    st.copy_(k.state)
    v, w = k.on()
    cu = [0, 4, 9]
    g.ssm_scan(v["x"], v["dt"], w["a"], v["b"], v["c"], head_dim=16, state_size=12, d=w["d"],
               dt_bias=w["dt_bias"], state=st, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(),
               slots=torch.tensor([2, 0], dtype=torch.int32).cuda(),
               resume=torch.tensor([True, True]).cuda())
    *_, new, nb, ns = k.want(spans=ref.ranges(9, cu), slots=[2, 0], resume=[True, True])
    check_state(st, new, nb, ns)
    assert (cache[:, :4] == 7.0).all() and (cache[:, 4 + 384:] == 7.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_garbage_behind_and_between_sequences(dtype):
    """NaN and infinities in rows of no sequence, or of a neighbour, reach nothing."""
    cu = [3, 40, 170]
    k = Case(180, 4, 64, 1, 128, dtype, slots=2)
    for t in (k.xbc, k.z):
        t[:3], t[170:] = float("nan"), float("inf")
        t[40:50] = float("nan")          # the second sequence's own rows
    st = k.state.cuda()
    got = k.run(cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), state=st)
    want, bound, size, new, nb, ns = k.want(spans=ref.ranges(180, cu))
    check(got[3:40], want[3:40], bound[3:40], size[3:40], dtype)
    assert torch.isnan(got[40:170].float()).all()
    check_state(st[:1], new[:1], nb[:1], ns[:1])
    assert torch.isnan(st[1]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("what", ["x", "b", "c", "dt"])
def test_bad_values_leave_the_rows_before_alone(dtype, bad, what):
    """A value that is not finite in one row: rows before it, other columns and
    other heads have what the definition gives, and it has the definition's
    infinities and NaN itself."""
    k = Case(300, 3, 64, 1, 24, dtype, slots=1, seed=4)
    row, col = 100, {"x": 64 + 5, "b": 3, "c": 7, "dt": 1}[what]
    k.views(k.xbc, k.z)[what][row, col] = bad
    st = k.state.cuda()
    got = k.run(state=st).double().cpu()
    want, bound, size, new, nb, ns = k.want(spans=[(0, 300)])
    fine = torch.isfinite(want)
    # (softplus of minus infinity is 0: nothing but a row without input)
    assert fine[:row].all() and (not fine.all() or (what, bad) == ("dt", -float("inf")))
    assert torch.equal(fine, torch.isfinite(got))
    tol = (bound + ref.rounding(want, dtype) + (size * torch.finfo(dtype).eps / 2
                                                if dtype != torch.float32 else 0)) * (1 + 2.0 ** -6)
    assert ((got - want).abs() <= tol)[fine].all()
    assert torch.equal(torch.isfinite(new), torch.isfinite(st.double().cpu()))


def test_offsets_that_do_not_ascend():
    """Nothing outside the buffers is touched whatever the offsets say."""
    rows = 700
    k = Case(rows, 2, 64, 1, 64, torch.bfloat16, slots=6)
    for cu in ([0, 700, 0, 700, 0, 700, 0], [-9, 5, 1 << 30, -(1 << 30), 650, 3, 700]):
        guard = torch.full((rows + 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        st = torch.cat([k.state, torch.full_like(k.state[:1], 7.0)]).cuda()
        k.run(cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), state=st[:6],
              out=guard[:rows])
        assert (guard[rows:] == 7.0).all() and (st[6:] == 7.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_same_bits_every_time(dtype):
    k = Case(1500, 4, 80, 2, 128, dtype, slots=1)
    first = None
    for _ in range(3):
        st = k.state.cuda()
        out = k.run(state=st)
        if first is None:
            first = (out, st)
        assert torch.equal(out, first[0]) and torch.equal(st, first[1])


def test_two_captured_graphs_and_streams():
    """Two graphs captured from the same call, replayed on two streams at once."""
    k = Case(3000, 2, 64, 1, 128, torch.bfloat16, slots=1)
    v, w = k.on()
    want = g.ssm_scan(v["x"], v["dt"], w["a"], v["b"], v["c"], head_dim=64, state_size=128,
                      d=w["d"], dt_bias=w["dt_bias"])
    runs = []
    for _ in range(2):
        s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        out = torch.empty_like(want)
        with torch.cuda.graph(graph, stream=s):
            g.ssm_scan(v["x"], v["dt"], w["a"], v["b"], v["c"], head_dim=64, state_size=128,
                       d=w["d"], dt_bias=w["dt_bias"], out=out)
        runs.append((s, graph, out))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, graph, out in runs:
            with torch.cuda.stream(s):
                out.zero_()
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for _, _, out in runs)


def test_refusals():
    k = Case(4, 2, 8, 1, 16, torch.float32)
    v, w = k.on()

    def call(**kw):
        a = {**v, **w, "head_dim": 8, "state_size": 16, **kw}
        return g.ssm_scan(a.pop("x"), a.pop("dt"), a.pop("a"), a.pop("b"), a.pop("c"), **a)

    call()
    for bad in (dict(head_dim=4), dict(state_size=5), dict(dt=v["dt"].bfloat16()),
                dict(b=v["b"][:2]), dict(a=w["a"].double()), dict(d=w["d"][:1]),
                dict(out=torch.empty(4, 16, dtype=torch.float16, device="cuda")),
                dict(slots=torch.zeros(1, dtype=torch.int32, device="cuda")),
                dict(state=torch.zeros(1, 2, 8, 15, device="cuda")),
                dict(state=torch.zeros(1, 2, 8, 16, dtype=torch.float16, device="cuda")),
                dict(state=torch.zeros(1, 2, 16, 8, device="cuda").transpose(2, 3)),
                dict(cu_seqlens=torch.zeros(2, dtype=torch.int64, device="cuda")),
                dict(state=torch.zeros(1, 2, 8, 16, device="cuda"), resume=torch.ones(1, device="cuda")),
                dict(state=torch.zeros(0, 2, 8, 16, device="cuda")),
                dict(dt=v["dt"].cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(dt_limits=(1.0, 0.0)), dict(out=v["x"])):
        with pytest.raises(g.GgrnError):
            call(**bad)
