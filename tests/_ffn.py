"""The feed-forward operators in 64 bits, with the largest error a correct
32-bit implementation can make, for the tests that compare with it.

Notation: u = 2^-24 is half a step of fp32 at 1.  A sum of n products in
fp32, in any order and with either rounding or truncation at each step, is
off by at most 2 n u sum|terms| to first order; `SUM` adds a few steps for
what surrounds the sum.  A result rounded to a type is off by half a step of
the type more (relative to the value: `torch.finfo(t).eps / 2`, and half the
smallest subnormal where that is larger).
"""

import math

import torch

U = 2.0 ** -24
F8 = torch.float8_e4m3fn
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, F8: 2.0 ** -4, torch.uint8: 2.0 ** -4}
LEAST = {torch.bfloat16: 0.0, torch.float32: 0.0, F8: 2.0 ** -10, torch.uint8: 2.0 ** -10}
# |act'| <= SLOPE and |act''| <= CURVE for every activation; relative and
# absolute error of the activation's own evaluation in fp32
SLOPE, CURVE = 1.13, 1.0
ACT_ERR = 16 * U


def sum_error(n, magnitude):
    return 2 * (n + 8) * U * magnitude


def phi(z):
    return 0.5 * torch.erfc(-z / math.sqrt(2.0))


def act(z, name):
    if name == "gelu":
        return z * phi(z)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    return z


def slope(z, name):
    if name == "gelu":
        return phi(z) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    if name == "relu":
        return (z > 0).to(z.dtype)
    return torch.ones_like(z)


def values(t):
    """An e4m3 byte tensor or any floating one in 64 bits."""
    return (t.view(F8) if t.dtype == torch.uint8 else t).to(torch.float64)


def mm(a, b):
    """a @ b^T in 64 bits (both contiguous: the right operand is never a transposed view)."""
    return torch.mm(a.contiguous(), b.t().contiguous())


def linear(x, w, bias=None, name=None, residual=None, xs=None, ws=None, out_scale=None, out=torch.bfloat16):
    """(y, its tolerance, preact, its tolerance)."""
    x, w = values(x), values(w)
    z, mag = mm(x, w), mm(x.abs(), w.abs())
    if xs is not None:
        z, mag = z * xs.double().reshape(-1, 1), mag * xs.double().abs().reshape(-1, 1)
    if ws is not None:
        z, mag = z * ws.double().reshape(1, -1), mag * ws.double().abs().reshape(1, -1)
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    ez = sum_error(x.shape[1], mag)
    y = act(z, name)
    ey = SLOPE * ez + ACT_ERR * z.abs()
    if residual is not None:
        y = y + residual.double()
        ey = ey + 2 * U * y.abs()
    if out in (F8, torch.uint8):
        f = 1.0 if out_scale is None else float(out_scale)
        y, ey = (y * f).clamp(-448, 448), ey * abs(f)
    return y, rounded(y, ey, out), z, rounded(z, ez, torch.bfloat16)


def rounded(y, e, dtype):
    """The tolerance of y, off by e before it was rounded to dtype."""
    return e + HALF_STEP[dtype] * (y.abs() + e) + LEAST[dtype]


def grad_input(dy, w, name=None, z=None):
    dy, w = dy.double(), w.double()
    wt = w.t().contiguous()
    g, mag = mm(dy, wt), mm(dy.abs(), wt.abs())
    e = sum_error(dy.shape[1], mag)
    if name is not None:
        s = slope(z.double(), name)
        g, e = g * s, SLOPE * e + ACT_ERR * (1 + z.double().abs()) * g.abs()
    return g, rounded(g, e, torch.bfloat16)


def grad_weight(dy, x, dtype=torch.bfloat16):
    a, b = dy.double().t().contiguous(), x.double().t().contiguous()
    g = mm(a, b)
    return g, rounded(g, sum_error(dy.shape[0], mm(a.abs(), b.abs())), dtype)


def column_sum(dy):
    return dy.double().sum(0), sum_error(dy.shape[0], dy.double().abs().sum(0))


def near(got, want, tol, what=""):
    got = values(got)
    bad = ~((got - want).abs() <= tol)
    bad &= ~(got.isnan() & want.isnan())
    if bool(bad.any()):
        at = [int(v) for v in bad.nonzero()[0]]
        raise AssertionError("%s: %d of %d values off, first at %s: got %r, want %r within %r"
                             % (what, int(bad.sum()), bad.numel(), at, float(got[tuple(at)]), float(want[tuple(at)]),
                                float(tol.expand_as(want)[tuple(at)])))


def inside_nan(t, left=3, right=5, rows=2):
    """The same matrix as a strided view in the middle of NaN."""
    big = torch.full((t.shape[0] + 2 * rows, t.shape[1] + left + right), 0x7F, dtype=torch.uint8, device=t.device) \
        .view(t.dtype) if t.element_size() == 1 else \
        torch.full((t.shape[0] + 2 * rows, t.shape[1] + left + right), math.nan, dtype=t.dtype, device=t.device)
    v = big[rows:rows + t.shape[0], left:left + t.shape[1]]
    v.copy_(t)
    return v


def edges(rows):
    """int32 offsets of groups of these row counts."""
    at = [0]
    for r in rows:
        at.append(at[-1] + r)
    return torch.tensor(at, dtype=torch.int32, device="cuda")
