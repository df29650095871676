"""layer_norm and layer_norm_backward against 64-bit forms.

Tolerances (u = 2^-24): each thread adds at most cols / 64 + 1 values and a
tree joins the threads, so a sum over a row is off by at most
(cols / 64 + 16) u sum|terms|; the values around it take a few steps of fp32
each, and a result is rounded once to its type."""

import math

import pytest

import _ffn as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = R.U


@pytest.fixture(scope="module")
def ec():
    import lossless_entropy_coding_amd as ec
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ec.lib()
    return ec


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def reference(x, w, b, eps):
    """mean, rstd, h in 64 bits and the errors fp32 can make of them."""
    x = x.double()
    n = x.shape[1]
    s = (n / 64 + 16) * U
    mean = x.mean(1, keepdim=True)
    e_mean = s * x.abs().mean(1, keepdim=True)
    d = x - mean
    var = (d * d).mean(1, keepdim=True)
    e_d = e_mean + U * (x.abs() + mean.abs())                      # of a centred value
    e_var = s * var + (2 * d.abs() * e_d + e_d * e_d).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    rel = (0.5 * e_var / (var + eps)).clamp(max=1.0) + 4 * U        # of rstd
    h = d * rstd
    e_h = e_d * rstd * (1 + rel) + h.abs() * (rel + 4 * U)
    y = h * w + b
    e_y = e_h * w.abs() + 4 * U * (h * w).abs() + 2 * U * (y.abs() + abs(b))
    return mean[:, 0], e_mean[:, 0] + U * mean.abs()[:, 0], rstd[:, 0], (rel * rstd)[:, 0], h, e_h, y, e_y


SHAPES = [(1, 1), (1, 2048), (2, 7), (3, 64), (5, 255), (4, 257), (33, 1000), (130, 2048), (7, 4099), (300, 72),
          (2, 16384), (3, 65536), (1030, 96), (64, 8192)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_layer_norm(ec, rows, cols, kind):
    print("norm %d %d %s" % (rows, cols, kind), flush=True)
    g = _gen(rows + cols)
    x = (torch.randn(rows, cols, generator=g, device="cuda") * 2 + 5).to(kind)
    wt = kind if cols % 2 else torch.float32
    w = (torch.randn(cols, generator=g, device="cuda") + 1).to(wt)
    b = torch.randn(cols, generator=g, device="cuda").to(wt)
    dy = torch.randn(rows, cols, generator=g, device="cuda").to(kind)
    dres = torch.randn(rows, cols, generator=g, device="cuda").to(kind)
    eps = 1e-5
    mean0, e_mean, rstd0, e_rstd, h, e_h, y0, e_y = reference(x, w.double(), b.double(), eps)
    for out, f in [(None, 1.0), (torch.float32, 1.0), (R.F8, 16.0), (torch.uint8, None)]:
        scale = torch.full((1,), f, device="cuda") if out == R.F8 else None
        y, mean, rstd = ec.layer_norm(x, w, b, eps, out_dtype=out, out_scale=scale)
        t = kind if out is None else out
        assert y.dtype == t
        ff = f or 1.0
        want = (y0 * ff).clamp(-448, 448) if t in (R.F8, torch.uint8) else y0
        R.near(y, want, R.rounded(want, e_y * ff, t), "y %s" % t)
        R.near(mean, mean0, e_mean, "mean")
        R.near(rstd, rstd0, e_rstd, "rstd")

    # backward, from the statistics as they were returned
    hh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    e_hh = 4 * U * (x.double().abs() + mean.double().abs()[:, None]) * rstd.double()[:, None]
    t = dy.double() * w.double()
    s = (cols / 64 + 16) * U
    mt, mth = t.mean(1, keepdim=True), (t * hh).mean(1, keepdim=True)
    e_mt = s * t.abs().mean(1, keepdim=True)
    e_mth = s * (t * hh).abs().mean(1, keepdim=True) + (t.abs() * e_hh).mean(1, keepdim=True)
    core = t - mt - hh * mth
    e_core = e_mt + e_hh * mth.abs() + (hh.abs() + e_hh) * e_mth + 4 * U * (t.abs() + mt.abs() + (hh * mth).abs())
    r = rstd.double()[:, None]
    for res in (dres, None):
        dx, dw, db = ec.layer_norm_backward(dy, x, mean, rstd, w, residual_grad=res)
        want = core * r + (res.double() if res is not None else 0)
        R.near(dx, want, R.rounded(want, e_core * r + 4 * U * (core * r).abs(), kind), "dx")
        terms = dy.double() * hh
        R.near(dw, terms.sum(0), R.sum_error(rows, terms.abs().sum(0)) + (dy.double().abs() * e_hh).sum(0), "dweight")
        R.near(db, dy.double().sum(0), R.sum_error(rows, dy.double().abs().sum(0)), "dbias")
        again = ec.layer_norm_backward(dy, x, mean, rstd, w, residual_grad=res)
        assert all(torch.equal(a, c) for a, c in zip((dx, dw, db), again))


@pytest.mark.parametrize("rows,cols", [(5, 100), (9, 2048), (70, 1000)])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("left", [0, 3, 8])
def test_strides_and_neighbours(ec, rows, cols, kind, left):
    print("norm strides %d %d %s %d" % (rows, cols, kind, left), flush=True)
    g = _gen(rows + left)
    right = 8 - cols % 8 if left == 8 else 5
    x0, dy0, dr0 = (torch.randn(rows, cols, generator=g, device="cuda").to(kind) for _ in range(3))
    x, dy, dr = (R.inside_nan(t, left, right) for t in (x0, dy0, dr0))
    back = torch.full((rows + 4, cols + left + right), 7.0, device="cuda").to(kind)
    out, keep = back[2:2 + rows, left:left + cols], back.clone()
    y, mean, rstd = ec.layer_norm(x, out=out)
    want, m2, r2 = ec.layer_norm(x0)
    assert torch.equal(out, want) and torch.equal(mean, m2) and torch.equal(rstd, r2)
    back[2:2 + rows, left:left + cols] = 7.0
    assert torch.equal(back, keep)
    dx, dw, db = ec.layer_norm_backward(dy, x, mean, rstd, residual_grad=dr, dx=out)
    wx, ww, wb = ec.layer_norm_backward(dy0, x0, mean, rstd, residual_grad=dr0)
    assert dx is out and torch.equal(out, wx) and torch.equal(dw, ww) and torch.equal(db, wb)
    back[2:2 + rows, left:left + cols] = 7.0
    assert torch.equal(back, keep)


def test_edges(ec):
    """No rows; a constant row (variance zero); rows far from zero; rows with infinity and NaN stay their own."""
    z = torch.empty(0, 64, device="cuda").bfloat16()
    y, mean, rstd = ec.layer_norm(z)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = ec.layer_norm_backward(z, z, mean, rstd)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()

    x = torch.full((3, 200), 3.25, device="cuda")
    b = torch.arange(200, device="cuda", dtype=torch.float32)
    y, mean, rstd = ec.layer_norm(x, None, b, 1e-5)
    assert (mean == 3.25).all() and torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=4 * U)
    assert torch.equal(y, b.expand(3, 200))

    g = _gen(3)
    x = torch.randn(6, 500, generator=g, device="cuda")
    far = x + 4096.0                                    # 24 bits leave 2^-12 steps: the variance must not cancel
    _, _, rstd = ec.layer_norm(far)
    want = (far.double().var(1, correction=0) + 1e-5) ** -0.5
    assert ((rstd.double() - want).abs() <= 1e-3 * want).all()
    clean, _, _ = ec.layer_norm(x)
    x[2, 7], x[4, 0] = math.nan, math.inf
    y, mean, _ = ec.layer_norm(x)
    for r in (0, 1, 3, 5):
        assert torch.equal(y[r], clean[r])
    assert y[2].isnan().all() and y[4].isnan().all() and mean[2].isnan()


def test_gradients_against_differences(ec):
    g = _gen(11)
    rows, cols, h = 3, 40, 1e-4
    x = torch.randn(rows, cols, generator=g, device="cuda")
    w = torch.randn(cols, generator=g, device="cuda")
    t = torch.randn(rows, cols, generator=g, device="cuda")
    _, mean, rstd = ec.layer_norm(x, w)
    dx, dw, db = ec.layer_norm_backward(t, x, mean, rstd, w)

    def value(xx, ww):
        m = xx.mean(1, keepdim=True)
        v = ((xx - m) ** 2).mean(1, keepdim=True)
        return float((t.double() * ((xx - m) / (v + 1e-5).sqrt() * ww)).sum())

    xd, wd = x.double(), w.double()
    scale = float(t.abs().sum())
    for i, j in [(0, 0), (1, 17), (2, 39)]:
        e = torch.zeros_like(xd)
        e[i, j] = h
        num = (value(xd + e, wd) - value(xd - e, wd)) / (2 * h)
        assert abs(num - float(dx[i, j])) <= 1e-6 * scale       # h^2 and 1e-16 / h are both below
    for j in (0, 20, 39):
        e = torch.zeros_like(wd)
        e[j] = h
        num = (value(xd, wd + e) - value(xd, wd - e)) / (2 * h)
        assert abs(num - float(dw[j])) <= 1e-6 * scale


def test_far_rows_and_graph(ec):
    g = _gen(2)
    rows, cols = 70, 128
    far = torch.empty((1 << 32) + (1 << 20), dtype=torch.bfloat16, device="cuda")
    step = ((1 << 32) // rows) // 8 * 8
    x, dy = far.as_strided((rows, cols), (step, 1)), far.as_strided((rows, cols), (step, 1), 1024)
    out = far.as_strided((rows, cols), (step, 1), 2048)
    x.copy_(torch.randn(rows, cols, generator=g, device="cuda")), dy.copy_(torch.randn(rows, cols, generator=g, device="cuda"))
    y, mean, rstd = ec.layer_norm(x, out=out)
    assert torch.equal(y, ec.layer_norm(x.contiguous())[0])
    got = ec.layer_norm_backward(dy, x, mean, rstd, dx=out)
    want = ec.layer_norm_backward(dy.contiguous(), x.contiguous(), mean, rstd)
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    xs, ds = x.contiguous(), dy.contiguous()

    def run():
        y, mean, rstd = ec.layer_norm(xs)
        return (y, mean, rstd) + ec.layer_norm_backward(ds, xs, mean, rstd)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for r in range(3):
        xs.copy_(torch.randn(rows, cols, generator=g, device="cuda"))
        graph.replay()
        eager = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), r
