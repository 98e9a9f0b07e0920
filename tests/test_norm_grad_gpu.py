"""Layer norm and the norms' backward passes on the GPU against their formulas in
64 bits."""
import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from tests import train_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
# (rows, width): teams of a warp, CTAs of one to four vectors a thread, rows of odd
# elements, and widths that no CTA holds
LN = [(1, 8), (5, 1), (33, 100), (700, 64), (2, 960), (9, 1001), (3, 3840), (2, 5120), (2, 9000),
      (2, 2051), (3, 17000), (1, 40000)]


def _tensor(gen, rows, width, dtype, pad=0, col=0, mean=0.0):
    return (torch.randn(rows, col + width + pad, generator=gen) + mean).to(dtype)[:, col:col + width]


def _on(t):
    """A copy on the GPU with the same strides and offset modulo 16 bytes."""
    base = torch.empty(t.shape[0], t.stride(0) if t.shape[0] > 1 else t._base.shape[1]
                       if t._base is not None else t.shape[1], dtype=t.dtype, device="cuda")
    col = t.storage_offset()
    view = base[:, col:col + t.shape[1]]
    view.copy_(t)
    return view


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,width", LN)
def test_layer_norm(rows, width, dtype):
    gen = torch.Generator().manual_seed(rows * 7 + width)
    x, dout = _tensor(gen, rows, width, dtype, mean=0.5), _tensor(gen, rows, width, dtype)
    w, b = 1 + 0.5 * torch.randn(width, generator=gen), torch.randn(width, generator=gen)
    for bias in (b, None):
        got = g.layer_norm(_on(x), w.cuda(), None if bias is None else bias.cuda(), eps=1e-3)
        want, bound = ref.layer_norm(x, w, bias, 1e-3)
        ref.assert_close(got, want, bound, dtype, "out")
    want = ref.layer_norm_backward(dout, x, w, 1e-3)
    got = g.layer_norm_backward(_on(dout), _on(x), w.cuda(), eps=1e-3)
    for n, v in zip(("dx", "dw", "db"), got):
        ref.assert_close(v, *want[n], dtype if n == "dx" else torch.float32, n)
    again = g.layer_norm_backward(_on(dout), _on(x), w.cuda(), eps=1e-3, bias=False)
    assert again[2] is None and all(torch.equal(u, v) for u, v in zip(got[:2], again[:2]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,col", [(8, 8), (4, 4), (3, 1), (2, 0)])
def test_layer_norm_of_strided_rows(pad, col, dtype):
    """Rows that begin at 16-byte, 8-byte and odd addresses; outputs into columns."""
    rows, width = 37, 264
    gen = torch.Generator().manual_seed(pad)
    x, dout = (_tensor(gen, rows, width, dtype, pad, col) for _ in range(2))
    w, b = (torch.randn(width, generator=gen) for _ in range(2))
    whole = torch.full((rows, col + width + pad), 7.0, dtype=dtype, device="cuda")
    out = whole[:, col:col + width]
    g.layer_norm(_on(x), w.cuda(), b.cuda(), eps=1e-5, out=out)
    ref.assert_close(out, *ref.layer_norm(x, w, b, 1e-5), dtype, "out")
    want = ref.layer_norm_backward(dout, x, w, 1e-5)
    got = g.layer_norm_backward(_on(dout), _on(x), w.cuda(), eps=1e-5, dx=out)
    for n, v in zip(("dx", "dw", "db"), got):
        ref.assert_close(v, *want[n], dtype if n == "dx" else torch.float32, n)
    assert (whole[:, :col] == 7.0).all() and (whole[:, col + width:] == 7.0).all()


def test_layer_norm_far_from_zero():
    """A mean a thousand times the deviation: squares of the differences, not of x."""
    gen = torch.Generator().manual_seed(0)
    x, dout = _tensor(gen, 5, 3840, torch.float32, mean=1000.0), _tensor(gen, 5, 3840, torch.float32)
    w = torch.ones(3840)
    ref.assert_close(g.layer_norm(x.cuda(), w.cuda(), eps=1e-5), *ref.layer_norm(x, w, None, 1e-5),
                     torch.float32)
    want = ref.layer_norm_backward(dout, x, w, 1e-5)
    for n, v in zip(("dx", "dw", "db"), g.layer_norm_backward(dout.cuda(), x.cuda(), w.cuda(),
                                                             eps=1e-5)):
        ref.assert_close(v, *want[n], torch.float32, n)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", [100, 1001, 3840])
def test_layer_norm_of_rows_of_one_value(width, dtype):
    """Sums of up to 2^12 times an 8-bit value are exact: nothing is left of the row."""
    x = torch.tensor([1.0, -3.0, 96.0, 0.0]).to(dtype)[:, None].expand(4, width).contiguous().cuda()
    w, b = torch.full((width,), 2.0, device="cuda"), torch.full((width,), 0.5, device="cuda")
    assert (g.layer_norm(x, w, b, eps=1e-6) == 0.5).all()


NORM = [(3, 7680, 960), (2, 5120, 5120), (700, 960, 8), (9, 4800, 100), (40, 4096, 128),
        (13, 1001, 77), (5, 1001, 1001), (6, 30, 3), (1, 64, 64), (2, 12288, 6144), (2, 4100, 2050),
        (1, 36000, 18000), (300, 96, 96)]


@pytest.mark.parametrize("dtype,mode", [(d, "mamba2") for d in DTYPES] +
                         [(d, "onnx") for d in DTYPES[1:]])
@pytest.mark.parametrize("rows,width,group", NORM)
def test_gated_norm(rows, width, group, dtype, mode):
    gen = torch.Generator().manual_seed(rows * 7 + width)
    dout, y, z = (_tensor(gen, rows, width, dtype) for _ in range(3))
    z[0, :2] = torch.tensor([8.0, -8.0]).to(dtype)
    w = 1 + 0.5 * torch.randn(width if mode == "mamba2" else group, generator=gen)
    if mode == "onnx":
        w = w.to(dtype)
    want = ref.norm_backward(dout, y, z, w, group, 1e-3, mode)
    got = g.backward(_on(dout), _on(y), _on(z), w.cuda(), group_size=group, eps=1e-3, mode=mode)
    for n, v in zip(("dy", "dgate", "dw"), got):
        ref.assert_close(v, *want[n], torch.float32 if n == "dw" else dtype, n)
    assert got[2].shape == w.shape


@pytest.mark.parametrize("pad,col", [(64, 0), (4, 4), (5, 3)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_norm_of_a_packed_projection(pad, col, dtype):
    """y and gate as columns of one tensor, their gradients as columns of another."""
    rows, width, group = 50, 400, 100
    gen = torch.Generator().manual_seed(pad)
    proj = torch.randn(rows, col + 2 * width + pad, generator=gen).to(dtype)
    dout = torch.randn(rows, width, generator=gen).to(dtype)
    w = torch.randn(width, generator=gen)

    def split(t):
        return t[:, col:col + width], t[:, col + width:col + 2 * width]

    want = ref.norm_backward(dout, *split(proj), w, group, 1e-5, "mamba2")
    whole = torch.full(proj.shape, 7.0, dtype=dtype, device="cuda")
    dy, dgate = split(whole)
    dev = proj.cuda()
    got = g.backward(dout.cuda(), *split(dev), w.cuda(), group_size=group, eps=1e-5, dy=dy,
                     dgate=dgate)
    for n, v in zip(("dy", "dgate", "dw"), got):
        ref.assert_close(v, *want[n], torch.float32 if n == "dw" else dtype, n)
    assert (whole[:, :col] == 7.0).all() and (whole[:, col + 2 * width:] == 7.0).all()


def test_the_onnx_scale_in_its_other_shapes():
    gen = torch.Generator().manual_seed(1)
    dout, y, z = (_tensor(gen, 6, 32, torch.float16).cuda() for _ in range(3))
    w = torch.randn(8, generator=gen).half().cuda()
    want = g.backward(dout, y, z, w, group_size=8, eps=1e-6, mode="onnx")
    for shape in ((1, 8), (8, 1)):
        got = g.backward(dout, y, z, w.reshape(shape), group_size=8, eps=1e-6, mode="onnx")
        assert got[2].shape == shape and torch.equal(got[2].reshape(8), want[2])


def test_no_rows():
    none = torch.zeros(0, 24, device="cuda")
    w = torch.ones(24, device="cuda")
    assert g.layer_norm(none, w, eps=1e-5).shape == (0, 24)
    dx, dw, db = g.layer_norm_backward(none, none, w, eps=1e-5)
    assert dx.shape == (0, 24) and (dw == 0).all() and (db == 0).all()
    dy, dz, dw = g.backward(none, none, none, w, group_size=8, eps=1e-5)
    assert dy.shape == (0, 24) and (dw == 0).all()


def test_nan_stays_in_its_row_and_group():
    gen = torch.Generator().manual_seed(0)
    x, dout = (_tensor(gen, 40, 960, torch.bfloat16).cuda() for _ in range(2))
    x[7, 100] = float("nan")
    w = torch.ones(960, device="cuda")
    bad = torch.isnan(g.layer_norm(x, w, eps=1e-5))
    assert bad[7].all() and int(bad.sum()) == 960
    bad = torch.isnan(g.layer_norm_backward(dout, x, w, eps=1e-5)[0])
    assert bad[7].all() and int(bad.sum()) == 960
    dy, dz, dw = g.backward(dout, x, dout, w, group_size=96, eps=1e-5)
    for t in (dy, dz):
        bad = torch.isnan(t)
        assert bad[7, 96:192].all() and int(bad.sum()) == 96
    assert torch.isnan(dw[96:192]).all() and int(torch.isnan(dw).sum()) == 96


def test_the_same_bits_every_time_and_when_captured():
    gen = torch.Generator().manual_seed(0)
    x, dout, z = (_tensor(gen, 3000, 960, torch.bfloat16).cuda() for _ in range(3))
    w = torch.randn(960, generator=gen).cuda()

    def both():
        return (g.layer_norm_backward(dout, x, w, eps=1e-5) +
                g.backward(dout, x, z, w, group_size=96, eps=1e-5))

    want = both()
    for _ in range(3):
        assert all(torch.equal(u, v) for u, v in zip(want, both()))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        got = both()
    for t in got:
        t.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, got))
