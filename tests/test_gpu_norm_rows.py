"""layer_norm and its backward pass with more rows than workgroups run at a
time: each takes several, loads the next while it works on one, uses its LDS
again and adds its rows' weight gradients up; the last pass is ragged.

Rows that run at a time: 4096 up to 512 columns (forward and backward), 4096
forward and 2048 backward up to 2048, 1024 up to 4096 (and forward up to
8192), 512 backward beyond, where rows are cut into slices of 8192 columns, and
256 forward beyond 8192."""

import pytest

import test_gpu_layer_norm as base

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

SHAPES = [(4099, 96), (9000, 7), (4101, 512), (5001, 2048), (2051, 1000), (4500, 1020), (2500, 2047), (1100, 4099), (1030, 4096),
          (1030, 8192), (600, 9000), (515, 16384), (530, 20001), (300, 40000)]


@pytest.fixture(scope="module")
def ec():
    import lossless_entropy_coding_amd as ec
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ec.lib()
    return ec


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_rows_in_turn(ec, rows, cols, kind):
    """Against the 64-bit form, with every output type, with and without the residual's gradient, twice the same bits."""
    base.test_layer_norm(ec, rows, cols, kind)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows,cols", [(4099, 96), (5001, 2048), (1100, 4099), (600, 9000)])
def test_bad_rows_stay_their_own(ec, rows, cols):
    """NaN and infinity in rows of one pass reach no row of another."""
    print("bad rows %d %d" % (rows, cols), flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, dy = (torch.randn(rows, cols, generator=g, device="cuda").bfloat16() for _ in range(2))
    clean, mean, rstd = base_norm = ec.layer_norm(x)
    dx0, _, _ = ec.layer_norm_backward(dy, x, mean, rstd)
    bad = [0, 5, rows // 2, rows - 1]
    xb = x.clone()
    xb[bad[0], 3], xb[bad[1], 0], xb[bad[2], cols - 1], xb[bad[3], 1] = (float("nan"), float("inf"), float("nan"), float("-inf"))
    y, m, r = ec.layer_norm(xb)
    dx, _, _ = ec.layer_norm_backward(dy, xb, m, r)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[bad] = False
    for got, want in zip((y, m, r), base_norm):
        assert torch.equal(got[keep], want[keep])
    assert torch.equal(dx[keep], dx0[keep])
    assert y[bad].isnan().all() and dx[bad].isnan().all()
