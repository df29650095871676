"""Outputs over inputs: what is refused (CPU), and that the rest gives the
same bits as outputs of their own."""

import pytest

torch = pytest.importorskip("torch")

INVAL = 1


@pytest.fixture(scope="module")
def ec():
    import os
    import lossless_entropy_coding_amd as ec
    if not os.path.exists(ec.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    ec.lib()
    return ec


X, DY, DX, S, WS = 0x1000_0000, 0x2000_0000, 0x3000_0000, 0x100, 0x4000_0000


def _grad(ec, x=X, xs=9000, dy=DY, ds=9000, dx=DX, dxs=9000, rows=64, cols=9000, dtype=1):
    return ec.lib().layer_norm_grad(dy, ds, x, xs, dtype, rows, cols, S, S, None, 3, None, 0, dx, dxs, None, None, WS, 1 << 30,
                                    None)


@pytest.mark.parametrize("kw", [
    dict(dx=X), dict(dx=DY), dict(dx=X + 2), dict(dx=X - 4096), dict(dx=X + 63 * 18000 + 17998), dict(dx=X, rows=1),
    dict(dx=DY, dxs=10000), dict(dx=DY + 8000 * 2, dxs=20000, ds=20000), dict(dx=X + 12000 * 4, dxs=20000, xs=20000, dtype=3),
    dict(dx=X, cols=8193), dict(dx=DY, cols=65536, ds=65536, dxs=65536, xs=65536)], ids=str)
def test_wide_rows_refuse_dx_over_what_they_read(ec, kw):
    assert _grad(ec, **kw) == INVAL


if not torch.cuda.is_available():                  # on a GPU these would be launched
    @pytest.mark.parametrize("kw", [
        dict(), dict(dx=X + 64 * 18000), dict(dx=X - 64 * 18000), dict(dx=X + 10000 * 2, dxs=20000, xs=20000),
        dict(dx=X + 11000 * 4, dxs=20000, xs=20000, dtype=3), dict(dx=X, cols=8192), dict(dx=DY, cols=100),
        dict(dx=X + 18000, rows=1), dict(dx=X, rows=0)], ids=str)
    def test_others_are_taken(ec, kw):
        """No argument is refused; without a GPU the launch fails (or there are no rows to launch for)."""
        assert _grad(ec, **kw) != INVAL


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(3, 64), (70, 1000), (5000, 96), (2100, 2048), (600, 8192)])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_norm_in_place(ec, rows, cols, kind):
    print("in place %d %d %s" % (rows, cols, kind), flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, dy, dres, w = (_randn(g, rows, cols, dtype=kind) for _ in range(4))
    w = w[0].contiguous()
    y0, mean, rstd = ec.layer_norm(x, w)
    want = ec.layer_norm_backward(dy, x, mean, rstd, w, residual_grad=dres)
    for over in range(3):
        a = [t.clone() for t in (dy, x, dres)]
        got = ec.layer_norm_backward(a[0], a[1], mean, rstd, w, residual_grad=a[2], dx=a[over])
        assert all(torch.equal(p, q) for p, q in zip(got, want)), over
    y, _, _ = ec.layer_norm(x, w, out=x)
    assert y is x and torch.equal(y, y0)


@pytest.mark.gpu
def test_wide_norm_in_place_is_refused(ec):
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = _randn(g, 20, 9000), _randn(g, 20, 9000)
    _, mean, rstd = ec.layer_norm(x)
    for over in (x, dy):
        with pytest.raises(ec.ECError):
            ec.layer_norm_backward(dy, x, mean, rstd, dx=over)
    dres = _randn(g, 20, 9000)                      # read where it is written only
    want = ec.layer_norm_backward(dy, x, mean, rstd, residual_grad=dres)
    got = ec.layer_norm_backward(dy, x, mean, rstd, residual_grad=dres, dx=dres)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    both = torch.empty(20, 18016, dtype=torch.bfloat16, device="cuda")      # side by side in the same rows
    both[:, :9000] = x
    got = ec.layer_norm_backward(dy, both[:, :9000], mean, rstd, dx=both[:, 9008:18008])
    assert torch.equal(got[0], ec.layer_norm_backward(dy, x, mean, rstd)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(1, 100, 64), (20, 300, 200), (70, 130, 520), (300, 257, 96), (520, 264, 9000)])
def test_products_over_the_residual_and_the_preact(ec, m, n, k):
    print("in place product %d %d %d" % (m, n, k), flush=True)
    g = torch.Generator(device="cuda").manual_seed(m)
    x, w, res, dy, z = _randn(g, m, k), _randn(g, n, k), _randn(g, m, n), _randn(g, m, n), _randn(g, m, k)
    want = ec.linear(x, w, act="silu", residual=res)
    assert torch.equal(ec.linear(x, w, act="silu", residual=res, out=res), want)
    want, _, _ = ec.linear_backward(dy, x, w, preact=z, act="gelu", need_dw=False, need_db=False)
    got, _, _ = ec.linear_backward(dy, x, w, preact=z, act="gelu", need_dw=False, need_db=False, dx=z)
    assert got is z and torch.equal(got, want)
