"""Refusals of the feed-forward operators, on the CPU: the C entry points
with bad arguments (they return before anything is launched), and the
binding's own checks."""

import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ec():
    import os
    import lossless_entropy_coding_amd as ec
    if not os.path.exists(ec.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    ec.lib()
    return ec


INVAL = 1


def _args(**kw):
    """Arguments that would be fine for m = 4, n = 8, k = 16 (the pointers are never read by the host)."""
    from lossless_entropy_coding_amd.ffn import _LinearArgs
    a = _LinearArgs()
    base = dict(m=4, n=8, k=16, dtype=1, out_dtype=1, x=0x10000, x_stride=16, w=0x20000, w_stride=16, y=0x30000,
                y_stride=8, dy=0x40000, dy_stride=8, dx=0x50000, dx_stride=16, dw=0x60000, dw_stride=16)
    base.update(kw)
    for key, v in base.items():
        setattr(a, key, v)
    return a


@pytest.mark.parametrize("bad", [
    dict(x=0), dict(w=0), dict(y=0), dict(x=0x10001), dict(y=0x30001), dict(x_stride=15), dict(w_stride=8), dict(y_stride=7),
    dict(m=1 << 31), dict(n=1 << 32), dict(k=1 << 40), dict(dtype=0), dict(dtype=3), dict(dtype=9), dict(out_dtype=0),
    dict(out_dtype=4), dict(act=4), dict(bias=0x1000, bias_dtype=2), dict(bias=0x1001, bias_dtype=1),
    dict(bias=0x1002, bias_dtype=3), dict(residual=0x1001, residual_stride=8), dict(residual=0x1000, residual_stride=7),
    dict(preact=0x1000, preact_stride=4), dict(x_scale=0x1000, x_scales=3), dict(x_scale=0x1002, x_scales=1),
    dict(w_scale=0x1000, w_scales=0), dict(w_scale=0x1000, w_scales=4), dict(out_scale=0x1000), dict(groups=2),
    dict(groups=5000, offsets=0x1000, w_group_stride=128), dict(groups=2, offsets=0x1000, w_group_stride=127),
    dict(groups=2, offsets=0x1002, w_group_stride=128), dict(workspace=0x1008), dict(status=0x1002),
], ids=str)
def test_linear_forward_refuses(ec, bad):
    assert ec.lib().linear_forward(ctypes.byref(_args(**bad)), None) == INVAL


@pytest.mark.parametrize("bad", [
    dict(dy=0), dict(w=0), dict(dx=0), dict(dtype=2), dict(act=1), dict(act=1, preact=0x1000, preact_stride=15),
    dict(dx_stride=15), dict(dy_stride=7), dict(dx=0x50001), dict(groups=1), dict(act=7)], ids=str)
def test_linear_grad_input_refuses(ec, bad):
    assert ec.lib().linear_grad_input(ctypes.byref(_args(**bad)), None) == INVAL


@pytest.mark.parametrize("bad", [
    dict(dy=0), dict(x=0), dict(out_dtype=2), dict(dw_stride=15), dict(dw=0x60001), dict(db=0x1002), dict(dtype=2),
    dict(groups=3, offsets=0x1000, dw_group_stride=100)], ids=str)
def test_linear_grad_weight_refuses(ec, bad):
    assert ec.lib().linear_grad_weight(ctypes.byref(_args(**bad)), None) == INVAL


def test_null_arguments(ec):
    L = ec.lib()
    for f in (L.linear_forward, L.linear_grad_input, L.linear_grad_weight):
        assert f(None, None) == INVAL
    assert L.linear_workspace_bytes(None, 0) == 0


def test_layer_norm_refuses(ec):
    L = ec.lib()
    X, Y, S = 0x10000, 0x20000, 0x30000

    def fwd(x=X, dtype=1, rows=4, cols=64, xs=64, w=None, b=None, wt=3, eps=1e-5, y=Y, ot=1, ys=64, sc=None, mean=S,
            rstd=S):
        return L.layer_norm_forward(x, dtype, rows, cols, xs, w, b, wt, eps, y, ot, ys, sc, mean, rstd, None)

    for bad in [dict(x=None), dict(y=None), dict(dtype=2), dict(cols=0), dict(cols=65537), dict(rows=1 << 31),
                dict(xs=63), dict(ys=63), dict(w=X, wt=2), dict(b=X + 1, wt=1), dict(eps=-1.0), dict(eps=float("nan")),
                dict(ot=0), dict(sc=S), dict(mean=S + 2), dict(x=X + 1)]:
        assert fwd(**bad) == INVAL, bad

    need = L.layer_norm_grad_workspace_bytes(4, 64)
    assert need > 0 and L.layer_norm_grad_workspace_bytes(4, 0) == 0

    def bwd(dy=X, ds=64, x=X, xs=64, dtype=1, rows=4, cols=64, mean=S, rstd=S, w=None, wt=3, dres=None, rs=0, dx=Y,
            dxs=64, dw=S, db=S, ws=X, n=need):
        return L.layer_norm_grad(dy, ds, x, xs, dtype, rows, cols, mean, rstd, w, wt, dres, rs, dx, dxs, dw, db, ws, n,
                                 None)

    for bad in [dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(dtype=2), dict(ds=8), dict(dxs=63),
                dict(dres=X, rs=63), dict(ws=None), dict(n=need - 1), dict(ws=X + 8), dict(w=X, wt=0), dict(cols=0),
                dict(dw=S + 1)]:
        assert bwd(**bad) == INVAL, bad


def test_binding_refuses_host_tensors_and_wrong_types(ec):
    x, w = torch.zeros(4, 16).bfloat16(), torch.zeros(8, 16).bfloat16()
    off = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ec.ECError):
        ec.linear(x, w)
    with pytest.raises(ec.ECError):
        ec.linear(x, None)
    with pytest.raises(ec.ECError):
        ec.grouped_linear(x, w[None], off)
    with pytest.raises(ec.ECError):
        ec.grouped_linear(x, w[None], None)
    with pytest.raises(ec.ECError):
        ec.linear_backward(torch.zeros(4, 8).bfloat16(), x, w)
    with pytest.raises(ec.ECError):
        ec.grouped_linear_backward(torch.zeros(4, 8).bfloat16(), x, w[None], None)
    with pytest.raises(ec.ECError):
        ec.layer_norm(x)
    with pytest.raises(ec.ECError):
        ec.layer_norm(x[0])
    with pytest.raises(ec.ECError):
        ec.layer_norm_backward(x, x, torch.zeros(4), torch.ones(4))


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu(ec):
    """Shapes, types, strides and devices that do not fit raise before any launch."""
    d = "cuda"
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    x, w = torch.zeros(4, 16, device=d, dtype=bf), torch.zeros(8, 16, device=d, dtype=bf)
    f = torch.zeros(8, device=d)
    off = torch.tensor([0, 4], dtype=torch.int32, device=d)
    bad = [
        lambda: ec.linear(x.float(), w), lambda: ec.linear(x, w.half()), lambda: ec.linear(x.to(f8), w),
        lambda: ec.linear(x, w[:, :8]), lambda: ec.linear(x.t(), w), lambda: ec.linear(x[:, ::2], w[:, ::2]),
        lambda: ec.linear(x, w, f[:4]), lambda: ec.linear(x, w, f.double()), lambda: ec.linear(x, w, act="tanh"),
        lambda: ec.linear(x, w, residual=x), lambda: ec.linear(x, w, x_scale=f[:2]), lambda: ec.linear(x, w, w_scale=f[:3]),
        lambda: ec.linear(x, w, out_scale=f[:1]), lambda: ec.linear(x, w, out_dtype=torch.float16),
        lambda: ec.linear(x, w, out=torch.zeros(4, 9, device=d, dtype=bf)), lambda: ec.linear(x.expand(4, 16)[None], w),
        lambda: ec.linear(x[:1].expand(4, 16), w), lambda: ec.linear(x, w.cpu()), lambda: ec.linear(x, w, f.cpu()),
        lambda: ec.grouped_linear(x, w, off), lambda: ec.grouped_linear(x, w[None], off.long()),
        lambda: ec.grouped_linear(x, w[None], off[:1]), lambda: ec.grouped_linear(x, w[None], off, f),
        lambda: ec.grouped_linear(x, w[None].expand(3, 8, 16), torch.zeros(4, dtype=torch.int32, device=d)),
        lambda: ec.grouped_linear(x, w[None], off, status=f),
        lambda: ec.linear_backward(x, x, w), lambda: ec.linear_backward(torch.zeros(4, 8, device=d), x, w),
        lambda: ec.linear_backward(torch.zeros(4, 8, device=d, dtype=bf), x, w, act="gelu"),
        lambda: ec.linear_backward(torch.zeros(4, 8, device=d, dtype=bf), x, w, dw_dtype=torch.float16),
        lambda: ec.layer_norm(x, f), lambda: ec.layer_norm(x.half()), lambda: ec.layer_norm(x, out_dtype=torch.float16),
        lambda: ec.layer_norm(x, torch.zeros(16, device=d), torch.zeros(16, device=d, dtype=bf)),
        lambda: ec.layer_norm_backward(x, x.float(), f[:4], f[:4]),
        lambda: ec.layer_norm_backward(x, x, f[:3], f[:4]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ec.ECError):
            call()
            pytest.fail("call %d was not refused" % i)
