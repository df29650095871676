"""The gated block against its 64-bit form: sizes from one row to several
tiles, types, strides, experts, and the backward pass."""

import pytest

torch = pytest.importorskip("torch")

import _training as tr  # noqa: E402
from _ffn import F8, edges, inside_nan, near, values  # noqa: E402

pytestmark = pytest.mark.gpu

SIZES = [  # m, k, n
    (1, 16, 8), (1, 1, 1), (1, 2048, 1024), (2, 33, 17), (16, 96, 16), (17, 100, 130), (32, 513, 24), (32, 2048, 4096),
    (33, 64, 65), (70, 130, 33), (64, 8192, 40), (130, 72, 130), (129, 1000, 513), (260, 520, 300), (513, 96, 257),
    (1024, 256, 2048), (1000, 64, 1999),
]


@pytest.fixture(scope="module")
def ec():
    import lossless_entropy_coding_amd as ec
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ec.lib()
    return ec


def _gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _factors(g, m, k, n, kind, groups=None):
    w_shape = (2 * n, k) if groups is None else (groups, 2 * n, k)
    if kind == "bf16":
        return _rand(g, m, k), _rand(g, *w_shape, scale=max(k, 1) ** -0.5)
    return (_rand(g, m, k, scale=8, dtype=torch.float32).clamp(-448, 448).to(F8),
            _rand(g, *w_shape, scale=64, dtype=torch.float32).clamp(-448, 448).to(F8))


@pytest.mark.parametrize("act", [None, "gelu", "silu", "relu"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(ec, size, act):
    m, k, n = size
    g = _gen(m + k + n)
    x, w = _factors(g, m, k, n, "bf16")
    bias = _rand(g, 2 * n, dtype=torch.float32)
    y, pre = ec.gated_linear(x, w, bias, act=act, save_preact=True)
    want, tol, z, ztol = tr.gated(x, w, bias, act)
    near(y, want, tol, "y")
    near(pre, z, ztol, "preact")
    near(ec.gated_linear(x, w, act=act), *tr.gated(x, w, None, act)[:2], "without bias")


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32, F8, torch.uint8], ids=str)
@pytest.mark.parametrize("size", [(1, 64, 40), (7, 2050, 130), (40, 200, 70), (300, 1040, 260), (1024, 512, 1024)], ids=str)
def test_forward_e4m3(ec, size, out):
    m, k, n = size
    g = _gen(1)
    x, w = _factors(g, m, k, n, "e4m3")
    xs, ws = torch.rand(m, generator=g, device="cuda") / 8, torch.rand(2 * n, generator=g, device="cuda") / (64 * k ** 0.5)
    os = torch.full((1,), 5.0, device="cuda") if out in (F8, torch.uint8) else None
    bias = _rand(g, 2 * n)
    y = ec.gated_linear(x.view(torch.uint8), w, bias, act="gelu", x_scale=xs, w_scale=ws, out_scale=os, out_dtype=out)
    assert y.dtype == out
    near(y, *tr.gated(x, w, bias, "gelu", xs, ws, os, out)[:2], "a scale a row and a column")
    one = torch.full((1,), 0.01, device="cuda")
    y = ec.gated_linear(x, w, act="silu", x_scale=one, w_scale=one, out_scale=os, out_dtype=out)
    near(y, *tr.gated(x, w, None, "silu", one, one, os, out)[:2], "one scale")


@pytest.mark.parametrize("size", [(1, 65, 9), (20, 100, 50), (90, 77, 131), (300, 264, 520)], ids=str)
def test_forward_strides(ec, size):
    """Rows at odd addresses in the middle of NaN, and outputs whose surroundings stay."""
    m, k, n = size
    g = _gen(2)
    x, w = _factors(g, m, k, n, "bf16")
    out = inside_nan(torch.zeros(m, n, dtype=torch.bfloat16, device="cuda"))
    pre = inside_nan(torch.zeros(m, 2 * n, dtype=torch.bfloat16, device="cuda"), left=1)
    whole = out._base
    y, p = ec.gated_linear(inside_nan(x), inside_nan(w, left=1), act="silu", out=out, preact=pre)
    assert y is out and p is pre
    want, tol, z, ztol = tr.gated(x, w, None, "silu")
    near(y, want, tol)
    near(p, z, ztol)
    keep = torch.ones_like(whole, dtype=torch.bool)
    keep[2:2 + m, 3:3 + n] = False
    assert bool(whole[keep].isnan().all())


def test_exact_values(ec):
    """Small whole numbers: every sum is exact, so that each result is the rounded one."""
    g = _gen(3)
    for m, k, n in [(1, 40, 12), (30, 64, 16), (130, 96, 72), (300, 200, 260)]:
        x = torch.randint(-2, 3, (m, k), generator=g, device="cuda").bfloat16()
        w = torch.randint(-2, 3, (2 * n, k), generator=g, device="cuda").bfloat16()
        z = tr.mm(x.double(), w.double())
        y, pre = ec.gated_linear(x, w, act="relu", save_preact=True, out_dtype=torch.float32)
        assert torch.equal(y.double(), z[:, :n].clamp(min=0) * z[:, n:])
        assert torch.equal(pre, z.bfloat16())
        dy = torch.randint(-1, 2, (m, n), generator=g, device="cuda").bfloat16()
        p = torch.randint(-2, 3, (m, 2 * n), generator=g, device="cuda").bfloat16()
        dz = torch.cat([dy.double() * p[:, n:].double() * (p[:, :n] > 0), dy.double() * p[:, :n].double().clamp(min=0)], 1)
        dx, dw, db = ec.gated_linear_backward(dy, x, w, p, act="relu", dw_dtype=torch.float32)
        assert torch.equal(dx, tr.mm(dz, w.double().t().contiguous()).bfloat16())
        assert torch.equal(dw.double(), tr.mm(dz.t().contiguous(), x.double().t().contiguous()))
        assert torch.equal(db.double(), dz.sum(0))


@pytest.mark.parametrize("m,k,n", [(0, 16, 8), (5, 0, 8), (5, 16, 0), (0, 0, 0)])
def test_empty(ec, m, k, n):
    x, w = torch.zeros(m, k, device="cuda").bfloat16(), torch.zeros(2 * n, k, device="cuda").bfloat16()
    bias = torch.full((2 * n,), 2.0, device="cuda")
    y, pre = ec.gated_linear(x, w, bias, act=None, save_preact=True)
    assert y.shape == (m, n) and bool((y == 4).all()) and bool((pre == 2).all())
    dx, dw, db = ec.gated_linear_backward(torch.ones(m, n, device="cuda").bfloat16(), x, w, pre, act=None)
    assert dx.shape == x.shape and bool((dx == 0).all()) and bool((dw == 0).all()) and bool((db == 2 * m).all())


def test_special_values(ec):
    """Infinities and NaN stay in their row; a gate of -inf under SiLU or GELU is as the formula has it, or NaN."""
    g = _gen(4)
    for m in (4, 70):
        x, w = _factors(g, m, 64, 48, "bf16")
        clean = ec.gated_linear(x, w)
        x[1, 3] = float("nan")
        x[2, 5] = float("inf")
        y = ec.gated_linear(x, w)
        rows = [i for i in range(m) if i not in (1, 2)]
        assert torch.equal(y[rows], clean[rows]) and bool(y[1].isnan().all())
        assert not bool(y[2].isfinite().any())


# ------------------------------------------------------------------ by expert


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,before,after", [([3, 0, 1], 0, 0), ([0, 0], 2, 5), ([40, 1, 0, 90], 3, 2), ([600, 300, 5], 0, 1),
                                               ([1] * 70, 1, 1), ([0, 0, 2000], 0, 0)], ids=str)
def test_grouped(ec, rows, before, after, kind):
    g = _gen(5)
    m, E, k, n = sum(rows) + before + after, len(rows), 136, 72
    off = edges(rows) + before
    x, w = _factors(g, m, k, n, kind, E)
    if kind == "bf16":
        x[:before] = float("nan")
        x[m - after:] = float("nan")
    ws = torch.rand(E, 2 * n, generator=g, device="cuda") / 64
    bias = _rand(g, E, 2 * n, dtype=torch.float32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, pre = ec.grouped_gated_linear(x, w, off, bias, act="gelu", w_scale=ws, save_preact=True, status=status)
    assert int(status) == 0
    at = off.tolist()
    for e in range(E):
        lo, hi = at[e], at[e + 1]
        want, tol, z, ztol = tr.gated(x[lo:hi], w[e], bias[e], "gelu", None, ws[e])
        near(y[lo:hi], want, tol, "expert %d" % e)
        near(pre[lo:hi], z, ztol, "expert %d" % e)
    assert bool((y[:before] == 0).all()) and bool((y[m - after:] == 0).all()) and bool((pre[:before] == 0).all())


@pytest.mark.parametrize("rows,before,after", [([3, 0, 1], 0, 0), ([0, 0], 2, 5), ([40, 1, 0, 90], 3, 2), ([600, 300, 5], 0, 1)],
                         ids=str)
def test_grouped_backward(ec, rows, before, after):
    g = _gen(6)
    m, E, k, n = sum(rows) + before + after, len(rows), 104, 37
    off = edges(rows) + before
    x, w = _factors(g, m, k, n, "bf16", E)
    dy, pre = _rand(g, m, n), _rand(g, m, 2 * n)
    for t in (x, dy, pre):
        t[:before] = float("nan")
        t[m - after:] = float("nan")
    dx, dw, db = ec.grouped_gated_linear_backward(dy, x, w, off, pre, act="silu")
    at = off.tolist()
    for e in range(E):
        s = slice(at[e], at[e + 1])
        wants = tr.gated_backward(dy[s], x[s], w[e], pre[s], "silu")
        for got, (want, tol), name in zip((dx[s], dw[e], db[e]), wants, ("dx", "dw", "db")):
            near(got, want, tol, "%s of expert %d" % (name, e))
    assert bool((dx[:before] == 0).all()) and bool((dx[m - after:] == 0).all())


def test_grouped_bad_offsets(ec):
    g = _gen(7)
    x, w = _factors(g, 40, 64, 24, "bf16", 3)
    dy, pre = _rand(g, 40, 24), _rand(g, 40, 48)
    for bad, as_if in [([0, 30, 20, 40], [0, 30, 30, 40]), ([-5, 10, 20, 99], [0, 10, 20, 40])]:
        off, good = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (bad, as_if))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = ec.grouped_gated_linear(x, w, off, status=status)
        assert int(status) == ec.S_BAD_OFFSETS and torch.equal(y, ec.grouped_gated_linear(x, w, good))
        status.zero_()
        got = ec.grouped_gated_linear_backward(dy, x, w, off, pre, status=status)
        assert int(status) == ec.S_BAD_OFFSETS
        for a, b in zip(got, ec.grouped_gated_linear_backward(dy, x, w, good, pre)):
            assert torch.equal(a, b)


# ------------------------------------------------------------------- backward


@pytest.mark.parametrize("act", [None, "gelu", "silu", "relu"])
@pytest.mark.parametrize("size", [(1, 16, 8), (1, 1, 1), (2, 33, 17), (17, 100, 130), (70, 130, 33), (129, 1000, 513), (513, 96, 257),
                                  (1024, 256, 1024)], ids=str)
def test_backward(ec, size, act):
    m, k, n = size
    g = _gen(m * k + n)
    x, w = _factors(g, m, k, n, "bf16")
    dy, pre = _rand(g, m, n), _rand(g, m, 2 * n, scale=2)
    got = ec.gated_linear_backward(dy, x, w, pre, act=act)
    for t, (want, tol), name in zip(got, tr.gated_backward(dy, x, w, pre, act), ("dx", "dw", "db")):
        near(t, want, tol, name)
    again = ec.gated_linear_backward(dy, x, w, pre, act=act)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_backward_parts(ec):
    """Each result alone, given buffers, fp32 weights' gradient, strided inputs."""
    g = _gen(8)
    m, k, n = 75, 90, 41
    x, w = _factors(g, m, k, n, "bf16")
    dy, pre = _rand(g, m, n), _rand(g, m, 2 * n)
    wants = tr.gated_backward(dy, x, w, pre, "silu", torch.float32)
    dx, dw, db = ec.gated_linear_backward(inside_nan(dy), inside_nan(x), inside_nan(w), inside_nan(pre, left=1),
                                          dw_dtype=torch.float32)
    for t, (want, tol), name in zip((dx, dw, db), wants, ("dx", "dw", "db")):
        near(t, want, tol, name)
    for i, name in enumerate(("dx", "dw", "db")):
        need = {"need_" + v: v == name for v in ("dx", "dw", "db")}
        one = ec.gated_linear_backward(dy, x, w, pre, dw_dtype=torch.float32, **need)
        assert [v is None for v in one] == [j != i for j in range(3)]
        assert torch.equal(one[i], (dx, dw, db)[i])
    out = inside_nan(torch.zeros(2 * n, k, device="cuda"))
    assert ec.gated_linear_backward(dy, x, w, pre, need_dx=False, need_db=False, dw=out)[1] is out
    assert torch.equal(out, dw)
    assert ec.gated_linear_backward(dy, x, w, pre, need_dx=False, need_dw=False, need_db=False) == (None, None, None)


def test_backward_by_differences(ec):
    """The gradient of sum(y c) along random directions, by differences of the 64-bit form."""
    g = _gen(9)
    m, k, n = 6, 24, 16
    x, w = _factors(g, m, k, n, "bf16")
    bias, c = _rand(g, 2 * n, dtype=torch.float32), _rand(g, m, n)
    for act in ("gelu", "silu", None):
        _, pre = ec.gated_linear(x, w, bias, act=act, save_preact=True)
        dx, dw, db = ec.gated_linear_backward(c, x, w, pre, act=act, dw_dtype=torch.float32)

        def value(x, w, b):
            z = tr.mm(x, w) + b
            return float((tr.act(z[:, :n], act) * z[:, n:] * c.double()).sum())

        x8, w8, b8 = x.double(), w.double(), bias.double()
        for which, grad in (("x", dx), ("w", dw), ("b", db)):
            v = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
            h = 1e-4
            args = {"x": x8, "w": w8, "b": b8}
            plus, minus = dict(args), dict(args)
            plus[which], minus[which] = args[which] + h * v, args[which] - h * v
            slope = (value(**plus) - value(**minus)) / (2 * h)
            # off by the roundings to bf16 of preact (through curvature), dz and dx: a few 2^-8 of the sum of magnitudes
            room = 8 * 2.0 ** -8 * float((grad.double() * v).abs().sum())
            assert abs(slope - float((grad.double() * v).sum())) <= room


# ------------------------------------------------------------ streams, graphs


def test_stream_and_graph(ec):
    g = _gen(10)
    x, w = _factors(g, 200, 136, 72, "bf16")
    dy = _rand(g, 200, 72)
    side = torch.cuda.Stream()

    def both():
        y, pre = ec.gated_linear(x, w, save_preact=True)
        return (y, pre) + ec.gated_linear_backward(dy, x, w, pre)

    want = both()
    torch.cuda.synchronize()
    y = ec.gated_linear(x, w, stream=side)
    side.synchronize()
    assert torch.equal(y, want[0])
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = both()
    for k in range(3):
        x.copy_(_rand(g, 200, 136))
        graph.replay()
        torch.cuda.synchronize()
        eager = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager)), "replay %d" % k


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("size", [(2048, 1600, 2048), (1500, 1607, 2051), (160, 520, 8200), (250, 1536, 4100)], ids=str)
def test_large_tiles(ec, size, kind):
    m, k, n = size
    g = _gen(13)
    x, w = _factors(g, m, k, n, kind)
    s = torch.full((1,), 1e-3, device="cuda") if kind == "e4m3" else None
    bias = _rand(g, 2 * n, dtype=torch.float32)
    for act in ("gelu", "silu", "relu", None):
        y, pre = ec.gated_linear(x, w, bias, act=act, w_scale=s, save_preact=True)
        want, tol, z, ztol = tr.gated(x, w, bias, act, None, s)
        near(y, want, tol, "y")
        near(pre, z, ztol, "preact")
    if kind == "bf16":
        dy, pre = _rand(g, m, n), _rand(g, m, 2 * n)
        got = ec.gated_linear_backward(dy, x, w, pre)
        for t, (want, tol), name in zip(got, tr.gated_backward(dy, x, w, pre, "silu"), ("dx", "dw", "db")):
            near(t, want, tol, name)


def test_large_tiles_grouped(ec):
    g = _gen(14)
    rows, k, n = [1900, 0, 700, 300], 1600, 1030
    m, off = sum(rows) + 5, edges(rows) + 3
    x, w = _factors(g, m, k, n, "bf16", len(rows))
    y = ec.grouped_gated_linear(x, w, off, act="gelu")
    dy, pre = _rand(g, m, n), _rand(g, m, 2 * n)
    dx, dw, db = ec.grouped_gated_linear_backward(dy, x, w, off, pre)
    at = off.tolist()
    for e in range(len(rows)):
        s = slice(at[e], at[e + 1])
        near(y[s], *tr.gated(x[s], w[e], None, "gelu")[:2])
        for got, (want, tol) in zip((dx[s], dw[e], db[e]), tr.gated_backward(dy[s], x[s], w[e], pre[s], "silu")):
            near(got, want, tol)
    assert bool((y[:3] == 0).all()) and bool((y[-2:] == 0).all())


def test_contraction_split(ec):
    """Few tiles and a long contraction: sums of parts, joined."""
    g = _gen(11)
    for m, k, n in [(48, 16384, 32), (40, 12000, 100), (130, 9000, 70)]:
        x, w = _factors(g, m, k, n, "bf16")
        near(ec.gated_linear(x, w, act="gelu"), *tr.gated(x, w, None, "gelu")[:2], str((m, k, n)))
        x, w = _factors(g, m, k, n, "e4m3")
        s = torch.full((1,), 1e-3, device="cuda")
        near(ec.gated_linear(x, w, act="gelu", w_scale=s), *tr.gated(x, w, None, "gelu", None, s)[:2], "e4m3")


def test_more_values_than_31_bits(ec):
    """Weights of more than 2^31 bytes: the second half begins far from the first."""
    n, k = 300_000, 2048
    g = _gen(12)
    w = torch.zeros(2 * n, k, device="cuda", dtype=torch.bfloat16)
    probe = torch.tensor([0, 1, n - 1, n // 2], device="cuda")
    for rows in (probe, probe + n):
        w[rows] = _rand(g, 4, k, scale=k ** -0.5)
    for m in (2, 70):
        x = _rand(g, m, k)
        y = ec.gated_linear(x, w, act=None)
        at = torch.cat([probe, probe + n])
        near(y[:, probe], *tr.gated(x, w[at], None, None)[:2])
        rest = torch.ones(n, dtype=torch.bool, device="cuda")
        rest[probe] = False
        assert bool((y[:, rest] == 0).all())
    assert values(y).shape == (70, n)
