"""The operators together, as examples/feed_forward.py runs them, and the
products at sizes whose tiles are the largest, whole and partial, or whose
contraction is split.  Tolerances as in _ffn."""

import importlib.util
import math
import os

import pytest

import _ffn as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F8 = R.F8


@pytest.fixture(scope="module")
def ec():
    import lossless_entropy_coding_amd as ec
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ec.lib()
    return ec


@pytest.fixture(scope="module")
def ff():
    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    t = torch.randn(shape, generator=g, device="cuda") * scale
    return (t.clamp(-448, 448) if dtype == F8 else t).to(dtype)


@pytest.mark.parametrize("rows", [1, 17, 300])
def test_serve(ec, ff, rows):
    """The stream changes nothing, and each step is right given what the step before stored."""
    print("serve %d" % rows, flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows)
    layer = ff.Layer(256, 1040, seed=rows)
    x = _randn(g, rows, 256)
    cb = ff.codebook(layer, _randn(g, 64, 256))
    y, coded, status = ff.serve(layer, cb, x)
    assert int(status) == 0 and coded > 0
    a = ff.activations(layer, x)
    direct = ec.linear(a, layer.w2_e4m3, layer.b2, residual=x, x_scale=layer.act_unscale, w_scale=layer.w2_scale)
    assert torch.equal(y, direct)
    h, _, _ = ec.layer_norm(x, layer.norm_weight, layer.norm_bias)
    want, tol, _, _ = R.linear(h, layer.w1, layer.b1, "gelu", out=torch.uint8, out_scale=32.0)
    R.near(a, want, tol, "activations")
    want, tol, _, _ = R.linear(a, layer.w2_e4m3, layer.b2, None, x, layer.act_unscale, layer.w2_scale)
    R.near(y, want, tol, "y")


def test_train(ec, ff):
    """Every gradient is that of the step it belongs to, given what was handed to it."""
    g = torch.Generator(device="cuda").manual_seed(4)
    layer = ff.Layer(264, 520, seed=4)
    x, dy = _randn(g, 130, 264), _randn(g, 130, 264, scale=0.05)
    y, grads = ff.train(layer, x, dy)
    h, mean, rstd = ec.layer_norm(x, layer.norm_weight, layer.norm_bias)
    a, z = ec.linear(h, layer.w1, layer.b1, act="gelu", save_preact=True)
    want, tol, _, _ = R.linear(a, layer.w2, layer.b2, None, x)
    R.near(y, want, tol, "y")
    R.near(grads["w2"], *R.grad_weight(dy, a), "dw2")
    R.near(grads["b2"], *R.column_sum(dy), "db2")
    dz, _, _ = ec.linear_backward(dy, a, layer.w2, preact=z, act="gelu", need_dw=False, need_db=False)
    R.near(dz, *R.grad_input(dy, layer.w2, "gelu", z), "dz")
    R.near(grads["w1"], *R.grad_weight(dz, h), "dw1")
    R.near(grads["b1"], *R.column_sum(dz), "db1")
    dh, _, _ = ec.linear_backward(dz, h, layer.w1, need_dw=False, need_db=False)
    want = ec.layer_norm_backward(dh, x, mean, rstd, layer.norm_weight, residual_grad=dy)
    assert all(torch.equal(p, q) for p, q in zip((grads["x"], grads["norm_weight"], grads["norm_bias"]), want))


def test_experts(ec, ff):
    g = torch.Generator(device="cuda").manual_seed(8)
    x, w1, b1 = _randn(g, 90, 128), _randn(g, 5, 72, 128, scale=0.1), _randn(g, 5, 72, dtype=torch.float32)
    y, choice = ff.serve_experts(x, _randn(g, 5, 128), w1, b1)
    for e in range(5):
        at = choice == e
        want, tol, _, _ = R.linear(x[at], w1[e], b1[e], "silu")
        R.near(y[at], want, tol, "expert %d" % e)


# whole and partial 256 x 256 tiles; a contraction split over tiles of each size
LARGE = [(4096, 4096, 64), (4090, 4082, 72), (3841, 4090, 100), (1030, 2050, 8200), (520, 264, 9000), (70, 130, 8192)]


@pytest.mark.parametrize("m,n,k", LARGE)
@pytest.mark.parametrize("kind", [torch.bfloat16, F8])
def test_linear_large(ec, m, n, k, kind):
    print("linear %d %d %d %s" % (m, n, k, kind), flush=True)
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    x, w = _randn(g, m, k, dtype=kind), _randn(g, n, k, dtype=kind)
    bias, res = _randn(g, n, dtype=torch.float32), _randn(g, m, n)
    xs, ws = torch.rand(m, generator=g, device="cuda") / math.sqrt(k), torch.rand(n, generator=g, device="cuda")
    y, z = ec.linear(x, w, bias, act="gelu", residual=res, x_scale=xs, w_scale=ws, save_preact=True)
    want, tol, zw, ztol = R.linear(x, w, bias, "gelu", res, xs, ws)
    R.near(y, want, tol, "y")
    R.near(z, zw, ztol, "preact")
    assert torch.equal(y, ec.linear(x, w, bias, act="gelu", residual=res, x_scale=xs, w_scale=ws))


@pytest.mark.parametrize("m,n,k", [(4090, 72, 4082), (72, 4090, 4090), (9000, 520, 264), (8192, 130, 70), (64, 8200, 300)])
def test_backward_large(ec, m, n, k):
    print("backward %d %d %d" % (m, n, k), flush=True)
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    dy, w, z = _randn(g, m, n, scale=0.1), _randn(g, n, k), _randn(g, m, k)
    x = R.act(z.double(), "gelu").bfloat16()
    dx, dw, db = ec.linear_backward(dy, x, w, preact=z, act="gelu", dw_dtype=torch.float32)
    R.near(dx, *R.grad_input(dy, w, "gelu", z), "dx")
    R.near(dw, *R.grad_weight(dy, x, torch.float32), "dw")
    R.near(db, *R.column_sum(dy), "db")
    again = ec.linear_backward(dy, x, w, preact=z, act="gelu", dw_dtype=torch.float32)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), again))


@pytest.mark.parametrize("rows", [[1000, 2300, 0, 1, 255, 257, 4000, 378], [1024] * 8], ids=str)
@pytest.mark.parametrize("n,k", [(1000, 520), (1024, 512)])
def test_grouped_large(ec, rows, n, k):
    print("grouped %s %d %d" % (rows, n, k), flush=True)
    g = torch.Generator(device="cuda").manual_seed(n)
    m, E = sum(rows), len(rows)
    x, w, z = _randn(g, m, k), _randn(g, E, n, k, scale=1 / math.sqrt(k)), _randn(g, m, k)
    bias, dy = _randn(g, E, n, dtype=torch.float32), _randn(g, m, n, scale=0.1)
    off = R.edges(rows)
    y = ec.grouped_linear(x, w, off, bias, act="gelu")
    dx, dw, db = ec.grouped_linear_backward(dy, x, w, off, preact=z, act="silu")
    at = 0
    for e, r in enumerate(rows):
        s = slice(at, at + r)
        want, tol, _, _ = R.linear(x[s], w[e], bias[e], "gelu")
        R.near(y[s], want, tol, "y of group %d" % e)
        R.near(dx[s], *R.grad_input(dy[s], w[e], "silu", z[s]), "dx of group %d" % e)
        R.near(dw[e], *R.grad_weight(dy[s], x[s]), "dw of group %d" % e)
        R.near(db[e], *R.column_sum(dy[s]), "db of group %d" % e)
        at += r


@pytest.mark.parametrize("kind", [torch.bfloat16, F8])
@pytest.mark.parametrize("m,n,k", [(1, 100, 1537), (4, 4111, 203), (19, 300, 777), (32, 5000, 95), (7, 17, 3)])
def test_few_rows_at_any_address(ec, kind, m, n, k):
    """Rows at odd addresses, ending inside a load, in the middle of NaN."""
    print("few rows %s %d %d %d" % (kind, m, n, k), flush=True)
    g = torch.Generator(device="cuda").manual_seed(n)
    x0, w0 = _randn(g, m, k, dtype=kind), _randn(g, n, k, dtype=kind)
    x, w = R.inside_nan(x0, 1, 4), R.inside_nan(w0, 3, 2)
    want, tol, _, _ = R.linear(x0, w0, out=torch.float32)
    R.near(ec.linear(x, w, out_dtype=torch.float32), want, tol, "y")
