"""linear, grouped_linear and their backward passes against 64-bit forms, at
sizes, strides, types and row groups where a product can go wrong.  The
tolerances are bounds of what rounding can do (see _ffn)."""

import math

import pytest

import _ffn as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F8 = R.F8
ACTS = [None, "gelu", "silu", "relu"]


@pytest.fixture(scope="module")
def ec():
    import lossless_entropy_coding_amd as ec
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ec.lib()
    return ec


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    t = torch.randn(shape, generator=g, device="cuda") * scale
    if dtype == F8:
        t = t.clamp(-448, 448)
    return t.to(dtype)


# (m, n, k): one, odd, whole and partial tiles of every size in use, long contractions, few rows of wide weights
SIZES = [(1, 1, 1), (1, 64, 64), (1, 2050, 96), (2, 48, 2048), (3, 5, 7), (5, 1024, 1000), (8, 16, 513), (16, 512, 4096),
         (17, 33, 1000), (31, 640, 160), (33, 256, 320), (48, 100, 8200), (64, 128, 256), (65, 2048, 512),
         (130, 257, 129), (127, 384, 64), (256, 512, 384), (300, 1024, 4096), (513, 640, 96), (1023, 520, 1000)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("kind", [torch.bfloat16, F8])
def test_linear_sizes(ec, m, n, k, kind):
    print("linear %d %d %d %s" % (m, n, k, kind), flush=True)
    g = _gen(m * 7 + n * 3 + k)
    x, w = _randn(g, m, k, dtype=kind), _randn(g, n, k, scale=1 / math.sqrt(k) if kind != F8 else 1.0, dtype=kind)
    name = ACTS[(m + n + k) % 4]
    bias = _randn(g, n, dtype=torch.float32) if n % 2 == 0 else None
    res = _randn(g, m, n) if k % 2 == 0 else None
    xs = ws = None
    if kind == F8:
        xs = torch.rand(m if m % 2 else 1, generator=g, device="cuda") + 0.5
        ws = (torch.rand(n if k % 3 else 1, generator=g, device="cuda") + 0.5) / math.sqrt(k)
    y, z = ec.linear(x, w, bias, act=name, residual=res, x_scale=xs, w_scale=ws, save_preact=True)
    want, tol, zw, ztol = R.linear(x, w, bias, name, res, xs, ws)
    R.near(y, want, tol, "y")
    R.near(z, zw, ztol, "preact")
    y2 = ec.linear(x, w, bias, act=name, residual=res, x_scale=xs, w_scale=ws)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("m,n,k", [(1, 96, 512), (7, 100, 72), (40, 256, 256), (300, 500, 200)])
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32, F8, torch.uint8])
def test_linear_outputs(ec, m, n, k, name, out):
    print("linear out %d %d %d %s %s" % (m, n, k, name, out), flush=True)
    g = _gen(n + k)
    x, w = _randn(g, m, k), _randn(g, n, k, scale=2 / math.sqrt(k))
    bias = _randn(g, n)                              # bfloat16 bias
    res = _randn(g, m, n)
    scale = torch.full((1,), 24.0, device="cuda") if out in (F8, torch.uint8) else None
    y = ec.linear(x, w, bias, act=name, residual=res, out_dtype=out, out_scale=scale)
    assert y.dtype == out
    want, tol, _, _ = R.linear(x, w, bias, name, res, out_scale=24.0 if scale is not None else None, out=out)
    R.near(y, want, tol, "y")


def test_e4m3_result_saturates_and_keeps_nan(ec):
    x = torch.tensor([[1.0] * 32, [-1.0] * 32, [float("nan")] + [1.0] * 31, [float("inf")] * 32, [0.0] * 32],
                     device="cuda").bfloat16()
    w = torch.full((40, 32), 100.0, device="cuda").bfloat16()
    y = ec.linear(x, w, out_dtype=torch.uint8)
    assert (y[0] == 0x7E).all() and (y[1] == 0xFE).all() and ((y[2] & 0x7F) == 0x7F).all()
    assert (y[3] == 0x7E).all() and (y[4] == 0).all()


@pytest.mark.parametrize("kind", [torch.bfloat16, F8])
@pytest.mark.parametrize("m,n,k", [(1, 40, 96), (9, 70, 250), (70, 130, 96), (150, 264, 520), (290, 300, 333)])
@pytest.mark.parametrize("left", [0, 3, 16])
def test_linear_strides_and_neighbours(ec, kind, m, n, k, left):
    """Views in the middle of NaN: aligned or not, nothing outside the view counts, and nothing outside the output
    is written."""
    print("strides %s %d %d %d %d" % (kind, m, n, k, left), flush=True)
    g = _gen(left + m)
    right = 16 if left == 16 else 5
    pad = (-k) % 16 if left == 16 else 0
    x0, w0 = _randn(g, m, k, dtype=kind), _randn(g, n, k, dtype=kind)
    x, w = R.inside_nan(x0, left, right + pad), R.inside_nan(w0, left, right + pad)
    res = R.inside_nan(_randn(g, m, n), left, right)
    back = torch.full((m + 4, n + left + right), 7.0, device="cuda").bfloat16()
    out, keep = back[2:2 + m, left:left + n], back.clone()
    zback = back.clone()
    pre = zback[2:2 + m, left:left + n]
    xs = torch.full((1,), 1 / math.sqrt(k), device="cuda")
    y, z = ec.linear(x, w, act="silu", residual=res, x_scale=xs, out=out, preact=pre)
    assert y is out and z is pre
    want, tol, zw, ztol = R.linear(x0, w0, None, "silu", res, xs)
    R.near(out, want, tol, "y")
    R.near(pre, zw, ztol, "preact")
    for t in (back, zback):
        t[2:2 + m, left:left + n] = 7.0
        assert torch.equal(t, keep)


@pytest.mark.parametrize("m,n,k", [(0, 8, 8), (4, 0, 8), (4, 8, 0), (300, 128, 0), (0, 0, 0)])
def test_linear_empty(ec, m, n, k):
    x, w = torch.empty(m, k, device="cuda").bfloat16(), torch.empty(n, k, device="cuda").bfloat16()
    bias = torch.arange(n, device="cuda", dtype=torch.float32)
    y, z = ec.linear(x, w, bias, save_preact=True)
    assert y.shape == (m, n)
    assert torch.equal(y, bias.bfloat16().expand(m, n)) and torch.equal(z, y)
    dy = torch.ones(m, n, device="cuda").bfloat16()
    dx, dw, db = ec.linear_backward(dy, x, w)
    assert dx.shape == (m, k) and dw.shape == (n, k) and db.shape == (n,)
    assert (db == m).all() and (dw == 0).all()
    if n == 0:
        assert (dx == 0).all()


def test_one_bad_row_stays_its_own(ec):
    """NaN and infinity in a row of x, or a row of w, reach no other row or column."""
    g = _gen(1)
    for m, n, k in [(20, 96, 128), (300, 320, 128)]:
        x, w = _randn(g, m, k), _randn(g, n, k)
        clean = ec.linear(x, w)
        x[3, 5], x[m - 1, 0], w[7, k - 1] = math.nan, math.inf, math.nan
        y = ec.linear(x, w)
        keep = torch.ones(m, n, dtype=torch.bool, device="cuda")
        keep[3], keep[m - 1], keep[:, 7] = False, False, False
        assert torch.equal(y[keep], clean[keep])
        assert y[3].isnan().all() and y[:, 7].isnan().all()


BACK = [(1, 1, 1), (1, 64, 128), (3, 5, 7), (17, 130, 33), (64, 64, 64), (100, 72, 264), (130, 257, 129), (256, 256, 256),
        (300, 520, 96), (513, 128, 640), (1000, 264, 392)]


@pytest.mark.parametrize("m,n,k", BACK)
@pytest.mark.parametrize("name", ACTS)
def test_linear_backward(ec, m, n, k, name):
    print("backward %d %d %d %s" % (m, n, k, name), flush=True)
    g = _gen(m + n + k)
    dy, w, z = _randn(g, m, n, scale=0.1), _randn(g, n, k), _randn(g, m, k, scale=1.5)
    x = R.act(z.double(), name).bfloat16()
    dt = torch.float32 if (m + n) % 2 else torch.bfloat16
    dx, dw, db = ec.linear_backward(dy, x, w, preact=z if name else None, act=name, dw_dtype=dt)
    R.near(dx, *R.grad_input(dy, w, name, z), "dx")
    R.near(dw, *R.grad_weight(dy, x, dt), "dw")
    R.near(db, *R.column_sum(dy), "db")
    again = ec.linear_backward(dy, x, w, preact=z if name else None, act=name, dw_dtype=dt)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), again))


@pytest.mark.parametrize("m,n,k", [(9, 72, 264), (70, 130, 96), (290, 300, 333)])
@pytest.mark.parametrize("left", [0, 3, 8])
def test_backward_strides_and_neighbours(ec, m, n, k, left):
    print("backward strides %d %d %d %d" % (m, n, k, left), flush=True)
    g = _gen(m + left)
    right = 8 if left == 8 else 5
    pn, pk = ((-n) % 8, (-k) % 8) if left == 8 else (0, 0)
    dy0, w0, x0, z0 = _randn(g, m, n), _randn(g, n, k), _randn(g, m, k), _randn(g, m, k)
    dy, w, x, z = (R.inside_nan(dy0, left, right + pn), R.inside_nan(w0, left, right + pk),
                   R.inside_nan(x0, left, right + pk), R.inside_nan(z0, left, right + pk))
    backx = torch.full((m + 4, k + left + right), 7.0, device="cuda").bfloat16()
    backw = torch.full((n + 4, k + left + right), 7.0, device="cuda")
    keepx, keepw = backx.clone(), backw.clone()
    dx, dw = backx[2:2 + m, left:left + k], backw[2:2 + n, left:left + k]
    ec.linear_backward(dy, x, w, preact=z, act="gelu", dx=dx, dw=dw)
    R.near(dx, *R.grad_input(dy0, w0, "gelu", z0), "dx")
    R.near(dw, *R.grad_weight(dy0, x0, torch.float32), "dw")
    for t, keep, r, c in ((backx, keepx, m, k), (backw, keepw, n, k)):
        t[2:2 + r, left:left + c] = 7.0
        assert torch.equal(t, keep)


def test_gradients_against_differences(ec):
    """Central differences of a scalar of the forward pass, in fp32 outputs, against the backward pass."""
    g = _gen(5)
    m, n, k, h = 6, 40, 24, 2.0 ** -6
    z, w, t = _randn(g, m, k), _randn(g, n, k, scale=0.3), _randn(g, m, n)
    x = R.act(z.double(), "gelu").bfloat16()
    dx, dw, db = ec.linear_backward(t, x, w, preact=z, act="gelu", dw_dtype=torch.float32)

    def value(zz, ww):  # sum(t * (gelu(z) w^T)) in 64 bits
        return float((t.double() * R.mm(R.act(zz, "gelu"), ww)).sum())

    zd, wd = z.double(), w.double()
    for i, j in [(0, 0), (2, 7), (5, 23), (3, 11)]:
        e = torch.zeros_like(zd)
        e[i, j] = h
        num = (value(zd + e, wd) - value(zd - e, wd)) / (2 * h)
        # central differences: h^2 / 6 |third derivative| (<= 2 for gelu) per unit of gradient; bf16 rounding of dx
        gsum = float((t.double()[i].abs() * wd[:, j].abs()).sum())
        assert abs(num - float(dx[i, j])) <= gsum * (h * h / 6 * 2 + 1e-5) + 2.0 ** -8 * abs(num)
    xs = x.double()
    for i, j in [(0, 0), (39, 23), (17, 5)]:
        num = float((t.double()[:, i] * xs[:, j]).sum())
        assert abs(num - float(dw[i, j])) <= 1e-5 * float((t.double()[:, i].abs() * xs[:, j].abs()).sum())


GROUPS = [[5], [0, 0, 3], [1, 1, 1, 1], [64, 0, 1, 63], [130, 7, 0, 257, 3], [0, 300, 0, 0, 40], [2] * 70,
          [0] * 66 + [20], [17, 40, 0, 33] * 5]


@pytest.mark.parametrize("rows", GROUPS, ids=lambda r: "%dx%d" % (len(r), sum(r)))
@pytest.mark.parametrize("kind", [torch.bfloat16, F8])
@pytest.mark.parametrize("n,k", [(64, 64), (200, 136), (33, 75), (512, 1024)])
def test_grouped_linear(ec, rows, kind, n, k):
    print("grouped %s %s %d %d" % (rows[:8], kind, n, k), flush=True)
    g = _gen(n + k + len(rows))
    m, E = sum(rows), len(rows)
    x = _randn(g, m, k, dtype=kind)
    w = _randn(g, E, n, k, scale=1 / math.sqrt(k) if kind != F8 else 1.0, dtype=kind)
    bias = _randn(g, E, n, dtype=torch.float32)
    ws = (torch.rand(E, n, generator=g, device="cuda") + 0.5) / math.sqrt(k) if kind == F8 else None
    res = _randn(g, m, n)
    off = R.edges(rows)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, z = ec.grouped_linear(x, w, off, bias, act="gelu", residual=res, w_scale=ws, save_preact=True, status=status)
    assert int(status) == 0
    at = 0
    for e, r in enumerate(rows):
        s = slice(at, at + r)
        want, tol, zw, ztol = R.linear(x[s], w[e], bias[e], "gelu", res[s], None, ws[e] if ws is not None else None)
        R.near(y[s], want, tol, "y of group %d" % e)
        R.near(z[s], zw, ztol, "preact of group %d" % e)
        at += r


@pytest.mark.parametrize("rows", GROUPS, ids=lambda r: "%dx%d" % (len(r), sum(r)))
@pytest.mark.parametrize("n,k", [(64, 64), (200, 136), (33, 75), (264, 520)])
def test_grouped_backward(ec, rows, n, k):
    print("grouped backward %s %d %d" % (rows[:8], n, k), flush=True)
    g = _gen(n + k + len(rows))
    m, E = sum(rows), len(rows)
    dy, w, z = _randn(g, m, n, scale=0.1), _randn(g, E, n, k), _randn(g, m, k)
    x = R.act(z.double(), "silu").bfloat16()
    dx, dw, db = ec.grouped_linear_backward(dy, x, w, R.edges(rows), preact=z, act="silu")
    at = 0
    for e, r in enumerate(rows):
        s = slice(at, at + r)
        R.near(dx[s], *R.grad_input(dy[s], w[e], "silu", z[s]), "dx of group %d" % e)
        R.near(dw[e], *R.grad_weight(dy[s], x[s]), "dw of group %d" % e)
        R.near(db[e], *R.column_sum(dy[s]), "db of group %d" % e)
        at += r


@pytest.mark.parametrize("offsets,m", [([4, 9, 9, 20], 30), ([0, 5, 3, 8], 10), ([-3, 2, 50, 60], 12),
                                       ([7, 7, 7, 7], 9), ([2147483647, -2147483648, 5, 6], 8), ([40, 90, 200, 300], 400)])
def test_rows_of_no_group_and_bad_offsets(ec, offsets, m):
    """Rows before the first and after the last offset get zeros; offsets that decrease or leave the rows are
    reported and count as their running maximum within [0, m]."""
    print("offsets %s of %d" % (offsets, m), flush=True)
    g = _gen(m)
    E, n, k = len(offsets) - 1, 72, 80
    x, w, bias = _randn(g, m, k), _randn(g, E, n, k), _randn(g, E, n)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, z = ec.grouped_linear(x, w, off, bias, save_preact=True, status=status)
    bad = any(v < 0 or v > m for v in offsets) or any(a > b for a, b in zip(offsets, offsets[1:]))
    assert int(status) == (ec.S_BAD_OFFSETS if bad else 0)
    at, clean = 0, []
    for v in offsets:
        at = max(at, min(max(v, 0), m))
        clean.append(at)
    status.zero_()
    dy = _randn(g, m, n)
    dx, dw, db = ec.grouped_linear_backward(dy, x, w, off, status=status)
    assert int(status) == (ec.S_BAD_OFFSETS if bad else 0)
    held = torch.zeros(m, dtype=torch.bool, device="cuda")
    for e in range(E):
        s = slice(clean[e], clean[e + 1])
        held[s] = True
        want, tol, _, _ = R.linear(x[s], w[e], bias[e])
        R.near(y[s], want, tol, "y")
        R.near(dx[s], *R.grad_input(dy[s], w[e]), "dx")
        R.near(dw[e], *R.grad_weight(dy[s], x[s]), "dw")
        R.near(db[e], *R.column_sum(dy[s]), "db")
    for t in (y, z, dx):
        assert (t[~held] == 0).all()


def test_far_offsets(ec):
    """Rows, groups and contraction rows more than 2^32 bytes apart."""
    g = _gen(9)
    m, n, k, E = 70, 136, 128, 2
    far = torch.empty((1 << 32) + (1 << 20), dtype=torch.bfloat16, device="cuda")   # 8 GiB
    step = ((1 << 32) // m) // 8 * 8
    x, dy = far.as_strided((m, k), (step, 1)), far.as_strided((m, n), (step, 1), 1024)
    w = far.as_strided((E, n, k), ((1 << 31) + 64, k, 1), 4096)
    x.copy_(_randn(g, m, k)), dy.copy_(_randn(g, m, n)), w.copy_(_randn(g, E, n, k))
    x0, dy0, w0 = x.contiguous(), dy.contiguous(), w.contiguous()
    off = torch.tensor([0, 30, m], dtype=torch.int32, device="cuda")
    y = ec.grouped_linear(x, w, off)
    dx, dw, db = ec.grouped_linear_backward(dy, x, w, off)
    y1 = ec.linear(x, w[1])
    dx1, dw1, db1 = ec.linear_backward(dy, x, w[1])
    want, tol, _, _ = R.linear(x0, w0[1])
    R.near(y1, want, tol, "y")
    R.near(dx1, *R.grad_input(dy0, w0[1]), "dx")
    R.near(dw1, *R.grad_weight(dy0, x0), "dw")
    R.near(db1, *R.column_sum(dy0), "db")
    for e, s in enumerate((slice(0, 30), slice(30, m))):
        want, tol, _, _ = R.linear(x0[s], w0[e])
        R.near(y[s], want, tol, "y")
        R.near(dx[s], *R.grad_input(dy0[s], w0[e]), "dx")
        R.near(dw[e], *R.grad_weight(dy0[s], x0[s]), "dw")
        R.near(db[e], *R.column_sum(dy0[s]), "db")
    out = far.as_strided((m, n), (step, 1), 1 << 14)
    assert torch.equal(ec.linear(x, w[1], out=out), y1)


@pytest.mark.parametrize("m", [3, 300])
def test_streams_and_graph(ec, m):
    """On a side stream, and captured into a graph that is replayed with new inputs between eager work."""
    g = _gen(m)
    n, k, E = 200, 301, 3                          # odd: the factors are padded in the workspace
    x, w, z, dy = _randn(g, m, k), _randn(g, E, n, k), _randn(g, m, k), _randn(g, m, n)
    off = torch.tensor([0, m // 3, m // 3, m], dtype=torch.int32, device="cuda")

    def step(stream=None):
        y = ec.linear(x, w[0], act="gelu", stream=stream)
        y2 = ec.grouped_linear(x, w, off, act="silu", stream=stream)
        b = ec.linear_backward(dy, x, w[1], preact=z, act="gelu", stream=stream)
        b2 = ec.grouped_linear_backward(dy, x, w, off, preact=z, act="relu", stream=stream)
        return (y, y2) + b + b2

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for r in range(3):
        x.copy_(_randn(g, m, k)), dy.copy_(_randn(g, m, n))
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), r
