"""layer_norm's statistics where a row's mean is large against its spread:
constant rows, whose sums round, and rows far from zero."""

import pytest

import _ffn as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = R.U
COLS = [1, 7, 333, 1000, 2047, 2048, 3001, 5000, 9000, 20001, 40000]


@pytest.fixture(scope="module")
def ec():
    import lossless_entropy_coding_amd as ec
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ec.lib()
    return ec


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("value", [1e6 + 0.1, -0.1, 1 / 3, 12345.678, 1e-20])
def test_constant_rows(ec, cols, value):
    """The values are all the same, so the distance from any mean near them is a whole number of their steps, and the
    sums of that are exact: the mean is the value, the result the bias, and the spread what eps leaves."""
    print("constant %d %g" % (cols, value), flush=True)
    for kind, rows in [(torch.float32, 3), (torch.float32, 1100), (torch.bfloat16, 3)]:
        x = torch.full((rows, cols), value, device="cuda").to(kind)
        b = torch.linspace(-2, 2, cols, device="cuda")
        y, mean, rstd = ec.layer_norm(x, None, b, 1e-5, out_dtype=torch.float32)
        assert (mean == x[:, 0].float()).all()
        assert ((rstd.double() - 1e-5 ** -0.5).abs() <= 8 * U * 1e-5 ** -0.5).all()
        assert torch.equal(y, b.expand(rows, cols))
        dx, dw, db = ec.layer_norm_backward(torch.ones_like(x), x, mean, rstd)
        assert (dw == 0).all() and (db == rows).all()


@pytest.mark.parametrize("cols", [c for c in COLS if c > 300])
@pytest.mark.parametrize("rows", [3, 1100])
@pytest.mark.parametrize("far", [1e3, 1e6])
def test_rows_far_from_zero(ec, rows, cols, far):
    """x - mean is exact to half a step of the mean (U |mean|); the first mean is off by at most (cols / 64 + 16) U |x|,
    and what is left of that after it is taken out by as many U of itself."""
    print("far %d %d %g" % (rows, cols, far), flush=True)
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(rows, cols, generator=g, device="cuda") * 3 + far
    y, mean, rstd = ec.layer_norm(x, eps=1e-5)
    xd = x.double()
    mean0 = xd.mean(1, keepdim=True)
    d = xd - mean0
    var = (d * d).mean(1, keepdim=True)
    s = (cols / 64 + 16) * U
    first = s * xd.abs().mean(1, keepdim=True)          # the first mean's error
    seen = d.abs() + first                              # a value less the first mean, exact to U of itself
    e_off = s * seen.mean(1, keepdim=True) + U * seen   # of the second, and of a value less it
    e_mean = e_off.amax(1) + 2 * U * mean0[:, 0].abs()
    e_var = s * (var + first * first) + 2 * (d.abs() * e_off).mean(1, keepdim=True) + 4 * U * (var + first * first)
    rel = 0.5 * e_var / (var + 1e-5) + 4 * U
    R.near(mean, mean0[:, 0], e_mean, "mean")
    rstd0 = (var + 1e-5) ** -0.5
    R.near(rstd, rstd0[:, 0], (rel * rstd0)[:, 0], "rstd")
    want = d * rstd0
    R.near(y, want, R.rounded(want, e_off * rstd0 * (1 + rel) + want.abs() * (rel + 4 * U), torch.float32), "y")
