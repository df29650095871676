"""The gated block, the loss and the weight update in 64 bits, with the largest
error a correct 32-bit implementation can make (notation as in ``_ffn``)."""

import math

import torch

import _ffn
from _ffn import ACT_ERR, CURVE, HALF_STEP, SLOPE, U, act, mm, rounded, slope, sum_error, values

BF16 = 2.0 ** -8


def gated(x, w, bias=None, name=None, xs=None, ws=None, out_scale=None, out=torch.bfloat16):
    """(y, its tolerance, preact, its tolerance)."""
    _, _, z, pre = _ffn.linear(x, w, bias, None, None, xs, ws)
    # z's own error, from its tolerance before the rounding to bf16
    ez = (pre - BF16 * z.abs()) / (1 + BF16)
    n = w.shape[0] // 2
    g, u, eg, eu = z[:, :n], z[:, n:], ez[:, :n], ez[:, n:]
    a = act(g, name)
    ea = SLOPE * eg + ACT_ERR * g.abs()
    y = a * u
    ey = ea * u.abs() + a.abs() * eu + ea * eu + 4 * U * y.abs()
    if out in (_ffn.F8, torch.uint8):
        f = 1.0 if out_scale is None else float(out_scale)
        y, ey = (y * f).clamp(-448, 448), ey * abs(f)
    return y, rounded(y, ey, out), z, pre


def gated_dz(dy, preact, name=None):
    """(dz, its error before it is rounded)."""
    dy, z = dy.double(), preact.double()
    n = dy.shape[1]
    g, u = z[:, :n], z[:, n:]
    dz = torch.cat([dy * u * slope(g, name), dy * act(g, name)], 1)
    # the activation's own error; its slope's, as in the product's backward pass
    e = torch.cat([(dy * u).abs() * ACT_ERR * (1 + g.abs()), dy.abs() * ACT_ERR * g.abs()], 1) + 4 * U * dz.abs()
    return dz, e


def gated_backward(dy, x, w, preact, name=None, dw_dtype=torch.bfloat16):
    """((dx, tolerance), (dw, tolerance), (db, tolerance))."""
    dz, e = gated_dz(dy, preact, name)
    r = e + BF16 * (dz.abs() + e)              # dz as the products see it
    wt, x = w.double().t().contiguous(), x.double()
    dx = mm(dz, wt)
    ex = mm(r, wt.abs()) + sum_error(dz.shape[1], mm(dz.abs() + r, wt.abs()))
    a, at, rt = dz.t().contiguous(), (dz.abs() + r).t().contiguous(), r.t().contiguous()
    xt = x.t().contiguous()
    dw = mm(a, xt)
    ew = mm(rt, xt.abs()) + sum_error(dz.shape[0], mm(at, xt.abs()))
    db = dz.sum(0)
    eb = e.sum(0) + sum_error(dz.shape[0], dz.abs().sum(0))
    return (dx, rounded(dx, ex, torch.bfloat16)), (dw, rounded(dw, ew, dw_dtype)), (db, eb)


def loss(x, w, target, ignore=-100):
    """(loss, tolerance, lse, tolerance, logits, their error)."""
    x, w = x.double(), w.double()
    m, n = x.shape[0], w.shape[0]
    l, e = mm(x, w), sum_error(x.shape[1], mm(x.abs(), w.abs()))
    lse = torch.logsumexp(l, 1)
    # Moving every logit by e moves lse by at most the largest e.  The sum of
    # exponentials: exp2 of a difference d is off by (3 |d| + 4) u of it, where
    # those far below the maximum weigh little, at most the spread of the
    # logits; up to 32 values are added one after the other in a lane, then
    # tiles (of 16 columns at least) over the lanes, each join a few u and the
    # step of the maximum again.
    spread = l.amax(1) - l.amin(1)
    el = e.amax(1) + U * (256 + n / 256 + 8 * spread + 4 * lse.abs())
    kept = (target != ignore) & (target >= 0) & (target < n)
    row = torch.arange(m, device=x.device)
    at = torch.where(kept, target, torch.zeros_like(target)).long()
    value = torch.where(kept, lse - l[row, at], torch.zeros_like(lse))
    tol = torch.where(kept, el + e[row, at] + 2 * U * value.abs(), torch.zeros_like(lse))
    return value, tol, lse, el, l, e


def loss_backward(dloss, x, w, target, ignore=-100, dw_dtype=torch.bfloat16):
    """((dx, tolerance), (dw, tolerance))."""
    _, _, lse, el, l, e = loss(x, w, target, ignore)
    x, w = x.double(), w.double()
    m, n = l.shape
    kept = (target != ignore) & (target >= 0) & (target < n)
    x = torch.where(kept[:, None], x, torch.zeros_like(x))
    row = torch.arange(m, device=x.device)[kept]
    p = torch.exp(l - lse[:, None])
    G = p.clone()
    G[row, target[kept].long()] -= 1
    scale = (dloss.double() * torch.ones(m, device=x.device, dtype=torch.float64)) * kept
    d = (l - lse[:, None]).abs()
    eg = p * (torch.expm1((e + el[:, None])) + U * (3 * d + 8)) + 4 * U * G.abs()
    G, eg = G * scale[:, None], eg * scale[:, None].abs()
    r = eg + BF16 * (G.abs() + eg)
    wt = w.t().contiguous()
    dx = mm(G, wt)
    ex = mm(r, wt.abs()) + sum_error(n, mm(G.abs() + r, wt.abs()))
    Gt, at, rt, xt = (v.t().contiguous() for v in (G, G.abs() + r, r, x))
    dw = mm(Gt, xt)
    ew = mm(rt, xt.abs()) + sum_error(m, mm(at, xt.abs()))
    return (dx, rounded(dx, ex, torch.bfloat16)), (dw, rounded(dw, ew, dw_dtype))


# ------------------------------------------------------------------------ AdamW

BLOCK = 256
M32 = 0xFFFFFFFF


def mix(x):
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & M32
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & M32
    return x ^ (x >> 16)


def random_shares(seed, step, first, n):
    """The random numbers in [0, 1) of m's and of v's rounding for n places from `first` on."""
    key = mix(torch.tensor(step ^ int(mix(torch.tensor(seed)))))
    at = torch.arange(first, first + n)
    r = mix((at & M32) ^ mix((at >> 32) ^ key))
    return (r & 0xFFFF).double() / 65536, (r >> 16).double() / 65536


def adamw(p, g, m, v, step, lr, betas, eps, decay, scale=1.0):
    """One step (the `step`-th) in 64 bits from values in 64 bits: {name: (value, error)} of p, m and v."""
    b1, b2 = betas
    d = g * scale
    m2 = b1 * m + (1 - b1) * d
    em = U * (3 * (b1 * m).abs() + 4 * ((1 - b1) * d).abs() + m2.abs())
    v2 = b2 * v + (1 - b2) * d * d
    ev = U * (3 * b2 * v + 6 * (1 - b2) * d * d + v2)
    c1, c2 = 1 - b1 ** step, 1 - b2 ** step
    below = (v2 / c2).sqrt() + eps
    change = lr * m2 / c1 / below
    # the corrections are off by a few u (exp(t log b) - 1 of an exponent off by 2 u of itself), v's root by half of v's
    # share of error, and each operation by u
    share = torch.where(v2 > 0, ev / v2, torch.zeros_like(v2))
    ech = change.abs() * (24 * U + share) + lr / c1 * em / below
    p2 = p * (1 - lr * decay) - change
    ep = ech + U * (4 * p.abs() + 2 * p2.abs())
    return {"p": (p2, ep), "m": (m2, em), "v": (v2, ev)}


def power(e):
    """2^e, exactly (pow is not, on the GPU)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def least_scale(top, most):
    """The least power of two, 2^-60 at least, that takes `top` to at most `most` (float64)."""
    e = torch.ceil(torch.log2((top / most).clamp(min=2.0 ** -60)))
    e = torch.where(top > most * power(e), e + 1, e)            # log2 rounded down
    e = torch.where(top <= most * power(e - 1), e - 1, e)       # or up
    return power(e.clamp(min=-60))


def steps_of(a):
    """The distance of e4m3 values around a in [0, 448]."""
    _, e = torch.frexp(a)
    return power((e - 1).clamp(min=-6) - 3)


def random_rounding(value, share, root):
    """The grid values (scaled) that `value` (of one or more whole blocks, float64) rounds to, the scale of each block,
    and how far the decision was from the other one (as a share of the distance)."""
    size = value.abs()
    top = size.view(-1, BLOCK).amax(1)
    scale = least_scale(top.sqrt() if root else top, 448.0)
    each = scale.repeat_interleave(BLOCK)
    a = size.sqrt() / each if root else size / each
    step = steps_of(a)
    low = torch.floor(a / step) * step
    if root:
        part = (a * a - low * low) / ((low + step) ** 2 - low * low)
        up = share < part
        margin = (share - part).abs()
    else:
        part = (a - low) / step
        up = part + share >= 1
        margin = (part + share - 1).abs()
    # next to a value of the grid the other side of it gives the same value: how far the value is from one
    near = torch.minimum(part, 1 - part)
    return (low + up * step) * (1.0 if root else value.sign()), scale, margin, near


def held(state, name):
    """The values that an e4m3 state stands for."""
    t, s = getattr(state, name), getattr(state, name + "_scale")
    x = values(t) * s.double().repeat_interleave(BLOCK)
    return x * x if name == "v" else x


__all__ = [k for k in dir() if not k.startswith("__")] + ["math", "CURVE", "HALF_STEP"]
