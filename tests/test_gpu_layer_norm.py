"""GPU parity of layer norm, forward and backward, against the float64 oracle.

Bars (u = 2^-24, float32's unit roundoff; v = 2^-8, bfloat16's, which holds 8 significant bits): a row's sums are added in a tree
over lanes and waves after at most 16 values a lane (rows of up to 16384), so statistics are off by
at most about (16 + 10) u of the sum of magnitudes, and an output by a few such errors: 64 u of the
largest value, 4e-6. A wider row's lane adds width / 1024 values. Outputs held in bfloat16 add their
own rounding, v of each value. The sums over n rows add n / (waves) terms a lane, at random signs an
error of about sqrt(n) u of their rms: sqrt(n) * 8 u of the column's root sum of squares."""
import numpy as np
import pytest
import torch

from oracle import block_ops as ref
from parity import case, to_np

pytestmark = pytest.mark.gpu

DEV = "cuda"
U, V = 2.0 ** -24, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def amd(gpu_lib):
    import recurrent_nets_amd
    return recurrent_nets_amd


def _draw(seed, rows, width, dtype, offset=0.3):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((rng.standard_normal((rows, width)) * 1.7 + offset).astype(np.float32)).to(dtype)
    g = torch.from_numpy(rng.standard_normal((rows, width)).astype(np.float32))
    w = torch.from_numpy((1 + 0.3 * rng.standard_normal(width)).astype(np.float32))
    b = torch.from_numpy((0.3 * rng.standard_normal(width)).astype(np.float32))
    return x, g, w, b


def _near(got, want, bf16, what, per_value=64 * U):
    got, want = to_np(got), np.asarray(want)
    assert got.shape == want.shape
    assert np.all(np.isfinite(got)), what
    if not got.size:
        return
    off = np.abs(got - want)
    bound = per_value * np.max(np.abs(want)) + (V * np.abs(want) if bf16 else 0.0)
    assert np.all(off <= bound), (what, float(np.max(off / np.maximum(bound, 1e-300))))


# one wave at each number of chunks, odd widths, 2 to 16 waves, rows wider than registers hold
WIDTHS = [1, 2, 7, 64, 100, 256, 257, 512, 1000, 1024, 1028, 1544, 2048, 4100, 8192, 16384, 16640]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("x_dt,y_dt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
def test_forward(amd, width, x_dt, y_dt):
    rows = 5 if width > 512 else 13
    x, _, w, b = _draw(width, rows, width, DT[x_dt])
    case(f"layer norm forward {rows} x {width} {x_dt} -> {y_dt}")
    y, mean, rstd = amd.layer_norm_forward(x.to(DEV), w.to(DEV), b.to(DEV), 1e-5, out_dtype=DT[y_dt], want_stats=True)
    torch.cuda.synchronize()
    assert y.dtype == DT[y_dt]
    want, m, r = ref.layer_norm(to_np(x), to_np(w), to_np(b), 1e-5)
    if width <= 2:  # the distance of two values from their mean is known to their own rounding
        scale = np.max(r) * np.max(np.abs(to_np(x))) * 8 * U
        assert np.max(np.abs(to_np(y) - want)) <= scale + (V if y_dt == "bf16" else 0) * np.max(np.abs(want))
        return
    _near(y, want, y_dt == "bf16", "y")
    _near(mean, m, False, "mean")
    _near(rstd, r, False, "rstd")


@pytest.mark.parametrize("width", WIDTHS[2:])
@pytest.mark.parametrize("x_dt,g_dt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
def test_backward(amd, width, x_dt, g_dt):
    rows = 37
    x, g, w, b = _draw(width + 1, rows, width, DT[x_dt])
    g = g.to(DT[g_dt])
    _, m, r = ref.layer_norm(to_np(x), None, None, 1e-5)
    mean, rstd = (torch.from_numpy(t.astype(np.float32)) for t in (m, r))
    case(f"layer norm backward {rows} x {width} {x_dt}, gradient {g_dt}")
    dx, dw, db = amd.layer_norm_backward(*(t.to(DEV) for t in (x, g, mean, rstd, w)))
    torch.cuda.synchronize()
    assert dx.dtype == x.dtype
    wx, ww, wb = ref.layer_norm_backward(to_np(x), to_np(g), to_np(mean), to_np(rstd), to_np(w))
    _near(dx, wx, x_dt == "bf16", "dx")
    root = np.sqrt(rows) * np.sqrt(rows) * 8 * U * 4  # terms of size up to about 4
    assert np.max(np.abs(to_np(dw) - ww)) <= root * 4
    assert np.max(np.abs(to_np(db) - wb)) <= root * 4


@pytest.mark.parametrize("rows", [1, 3, 5000])
def test_rows(amd, rows):
    """Fewer rows than workgroups, and more than one walk holds; no weight and no bias."""
    x, g, _, _ = _draw(rows, rows, 96, torch.float32)
    case(f"layer norm {rows} x 96, no weight")
    y, mean, rstd = amd.layer_norm_forward(x.to(DEV), want_stats=True)
    dx, dw, db = amd.layer_norm_backward(x.to(DEV), g.to(DEV), mean, rstd)
    torch.cuda.synchronize()
    want, m, r = ref.layer_norm(to_np(x))
    _near(y, want, False, "y")
    wx, ww, wb = ref.layer_norm_backward(to_np(x), to_np(g), to_np(mean), to_np(rstd))
    _near(dx, wx, False, "dx")
    assert np.max(np.abs(to_np(dw) - ww)) <= rows ** 0.5 * 64 * U * 16
    assert np.max(np.abs(to_np(db) - wb)) <= rows ** 0.5 * 64 * U * 16


def test_no_rows(amd):
    x = torch.empty((0, 40), device=DEV)
    y, mean, rstd = amd.layer_norm_forward(x, want_stats=True)
    assert y.shape == (0, 40) and mean.shape == (0,)
    dx, dw, db = amd.layer_norm_backward(x, x, mean, rstd)
    torch.cuda.synchronize()
    assert dx.shape == (0, 40) and bool((dw == 0).all()) and bool((db == 0).all())


def test_constant_and_far_rows(amd):
    """A constant row (variance 0: y = bias) and rows far from zero, whose variance the centred sum keeps."""
    x = torch.full((2, 300), 3.25)
    x[1] = 1000.0 + torch.arange(300) % 2
    w, b = torch.full((300,), 2.0), torch.full((300,), 0.5)
    case("layer norm of constant and far rows")
    y = amd.layer_norm_forward(x.to(DEV), w.to(DEV), b.to(DEV), 1e-5)
    torch.cuda.synchronize()
    want = ref.layer_norm(to_np(x), to_np(w), to_np(b))[0]
    assert bool((y[0] == 0.5).all())
    # the mean, about 1000, is exact to u 1000, half a variance's root away: relative 1000 u * 4
    assert np.max(np.abs(to_np(y[1]) - want[1])) <= 4 * 1000 * U * 4


def test_not_finite_stays_in_its_row(amd):
    x, _, w, b = _draw(9, 12, 333, torch.float32)
    clean = amd.layer_norm_forward(x.to(DEV), w.to(DEV), b.to(DEV))
    x[5, 7] = float("nan")
    x[8, 0] = float("inf")
    case("layer norm with NaN and infinity")
    y = amd.layer_norm_forward(x.to(DEV), w.to(DEV), b.to(DEV))
    torch.cuda.synchronize()
    keep = [i for i in range(12) if i not in (5, 8)]
    assert torch.equal(y[keep], clean[keep])
    assert bool(y[5].isnan().all()) and bool(y[8].isnan().any())


def test_leading_axes_streams_and_repeats(amd):
    """(B, T, d) input, a side stream, the same bits on every run, and views that are not 16-byte aligned."""
    x, g, w, b = _draw(21, 60, 128, torch.bfloat16)
    x3, g3, w, b = x.view(4, 15, 128).to(DEV), g.view(4, 15, 128).to(DEV), w.to(DEV), b.to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    case("layer norm on a side stream")
    y, mean, rstd = amd.layer_norm_forward(x3, w, b, want_stats=True, stream=s)
    first = amd.layer_norm_backward(x3, g3, mean, rstd, w, stream=s)
    again = amd.layer_norm_backward(x3, g3, mean, rstd, w, stream=s)
    torch.cuda.synchronize()
    assert y.shape == x3.shape and mean.shape == (4, 15)
    for p, q in zip(first, again):
        assert torch.equal(p, q)
    _near(y, ref.layer_norm(to_np(x3), to_np(w), to_np(b))[0], True, "y")
    off = torch.empty(60 * 128 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(60, 128)
    off.copy_(x)
    y2 = amd.layer_norm_forward(off, w, b)
    torch.cuda.synchronize()
    assert torch.equal(y2.view(4, 15, 128), y) or float((y2.view(4, 15, 128).float() - y.float()).abs().max()) <= V * float(y.float().abs().max())


def test_graph_replays(amd):
    x, g, w, b = (t.to(DEV) for t in _draw(31, 700, 250, torch.float32))
    y, mean, rstd = amd.layer_norm_forward(x, w, b, want_stats=True)
    dx, dw, db = (torch.empty_like(t) for t in (x, w, b))
    ws = torch.empty(amd.layer_norm.layer_norm_backward_workspace_bytes(700, 250), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    case("layer norm in a graph")
    with torch.cuda.graph(graph):
        amd.layer_norm_forward(x, w, b, out=y, mean=mean, rstd=rstd)
        amd.layer_norm_backward(x, g, mean, rstd, w, dx=dx, dweight=dw, dbias=db, workspace=ws)
    for i in range(3):
        x.mul_(1.0 + 0.25 * i)
        graph.replay()
        torch.cuda.synchronize()
        ey, em, er = amd.layer_norm_forward(x, w, b, want_stats=True)
        for got, want in zip((y, dx, dw, db), (ey,) + amd.layer_norm_backward(x, g, em, er, w)):
            assert torch.equal(got, want)
