"""Grouped products of 17 to 32 rows a group on average: row tiles of 32 where
the groups' columns fill the card, of 16 where they do not, with groups that
are empty, end inside a tile or take several."""

import math

import pytest

import _ffn as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F8 = R.F8
ROWS = [[20] * 32, [17, 31, 32, 16, 33, 0, 1, 40] * 4, [0] * 30 + [320, 320], [32] * 16, [24, 23, 25]]


@pytest.fixture(scope="module")
def ec():
    import lossless_entropy_coding_amd as ec
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ec.lib()
    return ec


@pytest.mark.parametrize("rows", ROWS, ids=lambda r: "%dx%d" % (len(r), sum(r)))
@pytest.mark.parametrize("kind", [torch.bfloat16, F8])
@pytest.mark.parametrize("n,k", [(300, 200), (513, 301)])
def test_few_rows_by_group(ec, rows, kind, n, k):
    print("few rows by group %s %s %d %d" % (rows[:8], kind, n, k), flush=True)
    g = torch.Generator(device="cuda").manual_seed(n + len(rows))
    m, E = sum(rows), len(rows)

    def randn(*shape, dtype=kind):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    x, w, bias, res = randn(m, k), randn(E, n, k), randn(E, n, dtype=torch.float32), randn(m, n, dtype=torch.bfloat16)
    ws = (torch.rand(E, n, generator=g, device="cuda") + 0.5) / math.sqrt(k)
    y, z = ec.grouped_linear(x, w, R.edges(rows), bias, act="silu", residual=res, w_scale=ws, save_preact=True)
    at = 0
    for e, r in enumerate(rows):
        s = slice(at, at + r)
        want, tol, zw, ztol = R.linear(x[s], w[e], bias[e], "silu", res[s], None, ws[e])
        R.near(y[s], want, tol, "y of group %d" % e)
        R.near(z[s], zw, ztol, "preact of group %d" % e)
        at += r
    assert torch.equal(y, ec.grouped_linear(x, w, R.edges(rows), bias, act="silu", residual=res, w_scale=ws))
