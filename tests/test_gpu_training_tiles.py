"""The gated block, the loss and the products' backward passes at sizes for
which the plan takes tiles and joins that small sizes do not reach: 256 x 256
tiles of either kind and 256 x 128 ones, whole and with a split contraction."""

import pytest

torch = pytest.importorskip("torch")

import _ffn  # noqa: E402
import _training as tr  # noqa: E402
from _ffn import F8, edges, inside_nan, near  # noqa: E402

pytestmark = pytest.mark.gpu

ACTS = ("gelu", "silu", "relu", None)


@pytest.fixture(scope="module")
def ec():
    import lossless_entropy_coding_amd as ec
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ec.lib()
    return ec


def _rand(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _codes(g, *shape, scale):
    return _rand(g, *shape, scale=scale, dtype=torch.float32).clamp(-448, 448).to(F8)


@pytest.mark.parametrize("m,n,k", [
    (1023, 4099, 1543), (500, 8200, 2048), (129, 16389, 1543),      # 256 x 256, four waves
    (200, 16500, 77), (129, 16500, 64),                             # 256 x 256, eight waves
    (129, 4100, 12000),                                             # four waves, split, joined
    (129, 1030, 12000),                                             # 256 x 128, split, joined
], ids=str)
def test_gated(ec, m, n, k):
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    x, w, bias = _rand(g, m, k), _rand(g, 2 * n, k, scale=k ** -0.5), _rand(g, 2 * n, dtype=torch.float32)
    for act in ACTS:
        y, pre = ec.gated_linear(x, w, bias, act=act, save_preact=True)
        want, tol, z, ztol = tr.gated(x, w, bias, act)
        near(y, want, tol, "y, %s" % act)
        near(pre, z, ztol, "preact, %s" % act)
        assert torch.equal(ec.gated_linear(x, w, bias, act=act), y)


@pytest.mark.parametrize("m,n,k", [
    (2049, 16389, 1543), (700, 8200, 64),                           # 256 x 256
    (129, 2048, 65536),                                             # split, joined
    (200, 8200, 4096), (3000, 300, 65536),                          # 256 x 128, whole and split
], ids=str)
def test_gated_e4m3(ec, m, n, k):
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    x, w = _codes(g, m, k, scale=8), _codes(g, 2 * n, k, scale=64)
    xs, ws = torch.rand(m, generator=g, device="cuda") / 8, torch.rand(2 * n, generator=g, device="cuda") / (64 * k ** 0.5)
    one = torch.full((1,), 1 / (512 * k ** 0.5), device="cuda")
    bias = _rand(g, 2 * n)
    for act, a, b in (("gelu", xs, ws), ("silu", None, one), ("relu", xs, one), (None, None, ws / 8)):
        y, pre = ec.gated_linear(x, w, bias, act=act, x_scale=a, w_scale=b, save_preact=True)
        want, tol, z, ztol = tr.gated(x, w, bias, act, a, b)
        near(y, want, tol, "y, %s" % act)
        near(pre, z, ztol, "preact, %s" % act)
    scale = torch.full((1,), 16.0, device="cuda")
    y = ec.gated_linear(x, w, act="gelu", x_scale=xs, w_scale=ws, out_scale=scale, out_dtype=F8)
    near(y, *tr.gated(x, w, None, "gelu", xs, ws, scale, F8)[:2], "e4m3")


@pytest.mark.parametrize("rows,n,k,kind", [([2100, 0, 1500, 400], 1030, 1600, "bf16"), ([5100, 3080], 4096, 4096, "e4m3")], ids=str)
def test_gated_by_expert(ec, rows, n, k, kind):
    g = torch.Generator(device="cuda").manual_seed(n)
    E, m, off = len(rows), sum(rows) + 5, edges(rows) + 3
    if kind == "bf16":
        x, w = _rand(g, m, k), _rand(g, E, 2 * n, k, scale=k ** -0.5)
        ws = None
    else:
        x, w = _codes(g, m, k, scale=8), _codes(g, E, 2 * n, k, scale=64)
        ws = torch.rand(E, 2 * n, generator=g, device="cuda") / (512 * k ** 0.5)
    bias = _rand(g, E, 2 * n, dtype=torch.float32)
    at = off.tolist()
    for act in ACTS:
        y, pre = ec.grouped_gated_linear(x, w, off, bias, act=act, w_scale=ws, save_preact=True)
        for e in range(E):
            s = slice(at[e], at[e + 1])
            want, tol, z, ztol = tr.gated(x[s], w[e], bias[e], act, None, None if ws is None else ws[e])
            near(y[s], want, tol, "expert %d, %s" % (e, act))
            near(pre[s], z, ztol, "preact of expert %d, %s" % (e, act))
        for rest in (y[:3], y[-2:], pre[:3], pre[-2:]):
            assert bool((rest == 0).all())


@pytest.mark.parametrize("m,n,k", [(129, 4096, 8200), (400, 803, 16500), (8192, 65, 8200), (1537, 200, 16500)], ids=str)
def test_gated_backward(ec, m, n, k):
    """Contractions over 2 n columns (dx), split and whole, and over m rows (dw), split and whole."""
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    x, w = _rand(g, m, k), _rand(g, 2 * n, k, scale=k ** -0.5)
    dy, pre = _rand(g, m, n), _rand(g, m, 2 * n)
    got = ec.gated_linear_backward(dy, x, w, pre, act="gelu")
    for t, (want, tol), name in zip(got, tr.gated_backward(dy, x, w, pre, "gelu"), ("dx", "dw", "db")):
        near(t, want, tol, name)


@pytest.mark.parametrize("m,n,k", [
    (1537, 400, 16500), (8192, 129, 8200),                          # dw: contraction m, whole and split
    (400, 1607, 16500), (129, 8192, 8200), (300, 33000, 1607),      # dx: contraction n, whole and split
], ids=str)
def test_products(ec, m, n, k):
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    dy, w, x = _rand(g, m, n), _rand(g, n, k), _rand(g, m, k)
    dx, dw, _ = ec.linear_backward(dy, x, w, need_db=False, dw_dtype=torch.float32)
    near(dx, *_ffn.grad_input(dy, w), "dx")
    near(dw, *_ffn.grad_weight(dy, x, torch.float32), "dw")
    again = ec.linear_backward(dy, x, w, need_db=False, dw_dtype=torch.float32)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("rows,n,k", [([2100, 0, 1500, 400], 1600, 2048), ([3000, 1200, 795], 2060, 1607), ([64, 4800, 136], 2060, 1607)],
                         ids=str)
def test_products_by_expert(ec, rows, n, k):
    g = torch.Generator(device="cuda").manual_seed(n)
    E, m, off = len(rows), sum(rows) + 5, edges(rows) + 3
    dy, x, w = _rand(g, m, n), _rand(g, m, k), _rand(g, E, n, k)
    dx, dw, _ = ec.grouped_linear_backward(dy, x, w, off, need_db=False)
    at = off.tolist()
    for e in range(E):
        s = slice(at[e], at[e + 1])
        near(dx[s], *_ffn.grad_input(dy[s], w[e]), "dx of expert %d" % e)
        near(dw[e], *_ffn.grad_weight(dy[s], x[s]), "dw of expert %d" % e)
    assert bool((dx[:3] == 0).all()) and bool((dx[-2:] == 0).all())


def _loss(m, n, k, seed, ignored):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, w = _rand(g, m, k), _rand(g, n, k, scale=2 * k ** -0.5)
    t = torch.randint(n, (m,), generator=g, device="cuda")
    t = torch.where(torch.rand(m, generator=g, device="cuda") < ignored, torch.full_like(t, -100), t)
    return x, w, t, torch.randn(m, generator=g, device="cuda")


@pytest.mark.parametrize("m,n,k", [
    (3000, 50001, 130),         # dx: contraction n, split; dw: contraction m
    (8192, 2000, 1030),         # dx whole; logits of long rows; m the last that counts its rows by itself
    (8192, 2000, 2048), (9001, 1601, 2050),
    (8, 16384, 136), (9, 16384, 136), (16, 16369, 40), (17, 20001, 2050), (32, 33000, 1000),    # few rows, and tiles
    (8192, 35001, 2048),        # two pieces, dx's sums carried from one to the other
], ids=str)
@pytest.mark.parametrize("ignored", [0.1, 0.9])
def test_loss(ec, m, n, k, ignored):
    x, w, t, dl = _loss(m, n, k, m + n + k, ignored)
    loss, lse = ec.linear_cross_entropy(x, w, t)
    want, tol, want_lse, tol_lse, _, _ = tr.loss(x, w, t)
    near(lse, want_lse, tol_lse, "lse")
    near(loss, want, tol, "loss")
    del want, tol, want_lse, tol_lse, _
    dx, dw = ec.linear_cross_entropy_backward(dl, x, w, t, lse)
    (wx, tx), (ww, tw) = tr.loss_backward(dl, x, w, t)
    near(dx, wx, tx, "dx")
    near(dw, ww, tw, "dw")
    assert bool((dx[t == -100] == 0).all())
    again = ec.linear_cross_entropy_backward(dl, x, w, t, lse)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("m,n,k", [(9, 16400, 65), (32, 17001, 71), (8, 16400, 65)], ids=str)
def test_loss_of_few_strided_rows(ec, m, n, k):
    """Rows at odd addresses in the middle of NaN: few rows read them in place, tiles from a copy."""
    x, w, t, dl = _loss(m, n, k, 3, 0.2)
    loss, lse = ec.linear_cross_entropy(inside_nan(x), inside_nan(w, left=1), t)
    want, tol, want_lse, tol_lse, _, _ = tr.loss(x, w, t)
    near(lse, want_lse, tol_lse, "lse")
    near(loss, want, tol, "loss")
    dx = inside_nan(torch.zeros(m, k, device="cuda").bfloat16())
    dw = inside_nan(torch.zeros(n, k, device="cuda"), left=1)
    ec.linear_cross_entropy_backward(dl, inside_nan(x), inside_nan(w, left=1), t, lse, dx=dx, dw=dw)
    (wx, tx), (ww, tw) = tr.loss_backward(dl, x, w, t, dw_dtype=torch.float32)
    near(dx, wx, tx, "dx")
    near(dw, ww, tw, "dw")
    for base, (rows, cols), left in ((dx._base, (m, k), 3), (dw._base, (n, k), 1)):
        keep = torch.ones_like(base, dtype=torch.bool)
        keep[2:2 + rows, left:left + cols] = False
        assert bool(base[keep].isnan().all())


@pytest.mark.parametrize("m", [8191, 8192, 8193, 20000])
def test_rows_without_a_target(ec, m):
    """Up to 8192 rows and beyond, where another launch finds their places: targets outside the vocabulary are reported and
    count as ignored, and what such rows hold reaches nothing."""
    x, w, t, dl = _loss(m, 300, 24, m, 0.3)
    t[0], t[m - 1] = 5, 6
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, lse = ec.linear_cross_entropy(x, w, t, status=status)
    want = ec.linear_cross_entropy_backward(dl, x, w, t, lse, status=status)
    assert int(status) == 0
    (wx, tx), (ww, tw) = tr.loss_backward(dl, x, w, t)
    near(want[0], wx, tx, "dx")
    near(want[1], ww, tw, "dw")
    for at in (1, 1023, 1024, 8190, m - 2):
        for bad in (300, -1, 1 << 40, -(1 << 63)):
            wrong, ignored = t.clone(), t.clone()
            wrong[at], ignored[at] = bad, -100
            status.zero_()
            got = ec.linear_cross_entropy_backward(dl, x, w, wrong, lse, status=status)
            assert int(status) == ec.S_BAD_TARGET
            for a, b in zip(got, ec.linear_cross_entropy_backward(dl, x, w, ignored, lse)):
                assert torch.equal(a, b)
    none = t == -100
    assert bool(none[::64].any())
    x[none] = float("nan")
    x[none.nonzero()[::3, 0]] = float("inf")
    dl[none], lse[none] = float("nan"), float("inf")
    for a, b in zip(ec.linear_cross_entropy_backward(dl, x, w, t, lse), want):
        assert torch.equal(a, b)
    t.fill_(-100)
    for a in ec.linear_cross_entropy_backward(dl, x, w, t, lse):
        assert bool((a == 0).all())


def test_loss_of_few_rows_in_a_graph(ec):
    """Captured where tiles are taken, with another number of rows that have a target in each replay."""
    x, w, t, dl = _loss(24, 16500, 136, 5, 0.2)

    def both():
        loss, lse = ec.linear_cross_entropy(x, w, t)
        return (loss, lse) + ec.linear_cross_entropy_backward(dl, x, w, t, lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = both()
    for k, ignored in enumerate((0.0, 0.5, 1.0, 0.1)):
        nx, _, nt, ndl = _loss(24, 16500, 136, 10 + k, ignored)
        for to, new in ((x, nx), (t, nt), (dl, ndl)):
            to.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        eager = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager)), "replay %d" % k


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("k", [1, 31, 77, 2050, 4095, 4096, 4111])
@pytest.mark.parametrize("m", [1, 2, 4, 5])
def test_gated_few_rows_many_columns(ec, m, k, kind):
    """Up to four rows by 512 and more workgroups' columns share the waves by half (in e4m3 from 4096
    values on); lengths that end inside a load."""
    n = 8200
    g = torch.Generator(device="cuda").manual_seed(m * k)
    if kind == "bf16":
        x, w = _rand(g, m, k), _rand(g, 2 * n, k, scale=k ** -0.5)
        xs = ws = None
    else:
        x, w = _codes(g, m, k, scale=8), _codes(g, 2 * n, k, scale=64)
        xs, ws = torch.rand(m, generator=g, device="cuda") / 8, torch.rand(2 * n, generator=g, device="cuda") / (64 * k ** 0.5)
    bias = _rand(g, 2 * n, dtype=torch.float32)
    for act in ACTS:
        y, pre = ec.gated_linear(x, w, bias, act=act, x_scale=xs, w_scale=ws, save_preact=True)
        want, tol, z, ztol = tr.gated(x, w, bias, act, xs, ws)
        near(y, want, tol, "y, %s" % act)
        near(pre, z, ztol, "preact, %s" % act)
    out = torch.full((m, n + 3), float("nan"), dtype=torch.float32, device="cuda")
    ec.gated_linear(x, w, act="silu", x_scale=xs, w_scale=ws, out=out[:, 2:n + 2])
    near(out[:, 2:n + 2], *tr.gated(x, w, None, "silu", xs, ws, out=torch.float32)[:2], "inside a wider buffer")
    assert bool(out[:, :2].isnan().all()) and bool(out[:, n + 2:].isnan().all())
