"""The activations' own accuracy, far into their tails, in fp32 results.

z comes in whole through the bias (fp32, added to a sum of zeros), so nothing
but the activation is measured.  Tolerances, with u = 2^-24: the exponential
is off by the rounding of its exponent, z^2 / 2 (or z) times two roundings and
that of a constant, 2.5 u in all; the polynomial, the reciprocal, the
exponential itself and the products around them by 20 u together (a fit of
2.5 u, eight steps of Horner's rule at most 8 u more, 2 u each for the
reciprocal and the exponential, the rest for the products).  Below 2^-126 a
hardware exponential is zero."""

import math

import pytest

import _ffn as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = R.U
LEAST = 16 * 2.0 ** -126


@pytest.fixture(scope="module")
def ec():
    import lossless_entropy_coding_amd as ec
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ec.lib()
    return ec


def _sweep():
    z = torch.cat([torch.linspace(-14, 6, 20001), -torch.logspace(-6, 1, 1500), torch.logspace(-6, 2, 1500),
                   torch.tensor([0.0, -0.0, 1e18, -1e18, 1e30, -1e30, 3e38, -3e38])]).float()
    return z.cuda()


@pytest.mark.parametrize("name", ["gelu", "silu", "relu"])
@pytest.mark.parametrize("rows", [1, 40, 300])
def test_forward_keeps_relative_accuracy(ec, name, rows):
    print("activation %s %d" % (name, rows), flush=True)
    z = _sweep()
    x, w = (torch.zeros(s, 16, dtype=torch.bfloat16, device="cuda") for s in (rows, len(z)))
    y = ec.linear(x, w, z, act=name, out_dtype=torch.float32)
    zd = z.double()
    want = R.act(zd, name)
    rel = {"gelu": 20 * U + 2.5 * U * zd * zd / 2, "silu": 20 * U + 2.5 * U * zd.abs(), "relu": 0 * zd}[name]
    rel = torch.where(zd > 0, 20 * U, rel) if name != "relu" else rel
    R.near(y, want.expand(rows, -1), (rel.clamp(max=1.0) * want.abs() + LEAST).expand(rows, -1), name)


def slope_parts(z, name):
    """act'(z) and the sum of the magnitudes it is made of, each with the relative accuracy above."""
    if name == "gelu":
        p, q = R.phi(z), z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return p + q, p.abs() + q.abs()
    s = torch.sigmoid(z)
    q = z * s * (1 - s)
    return s + q, s + q.abs()


@pytest.mark.parametrize("name", ["gelu", "silu"])
def test_slope_keeps_relative_accuracy(ec, name):
    """dx = (dy w) act'(z) with dy w = 1, for every bf16 z of the range; one rounding to bf16."""
    print("slope %s" % name, flush=True)
    z = _sweep().bfloat16()
    z = torch.unique(z[z.float().abs() < 100])[None]
    k = z.shape[1]
    dy = torch.ones(40, 1, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(1, k, dtype=torch.bfloat16, device="cuda")
    dx, _, _ = ec.linear_backward(dy, z.expand(40, k).contiguous(), w, preact=z.expand(40, k).contiguous(), act=name,
                                  need_dw=False, need_db=False)
    zd = z.double()
    want, mag = slope_parts(zd, name)
    grow = zd * zd / 2 if name == "gelu" else zd.abs()
    e = mag * (20 * U + 2.5 * U * grow).clamp(max=1.0) + LEAST
    R.near(dx, want.expand(40, k), R.rounded(want, e, torch.bfloat16).expand(40, k), name)
