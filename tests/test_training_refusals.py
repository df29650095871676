"""Refusals of the gated block, the loss and the weight update, on the CPU:
the C entry points with bad arguments (they return before anything is
launched), and the binding's own checks."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

INVAL, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def ec():
    import os
    import lossless_entropy_coding_amd as ec
    if not os.path.exists(ec.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    ec.lib()
    return ec


def _gated(**kw):
    """Arguments that would be fine for m = 4, n = 8, k = 16 (the pointers are never read by the host)."""
    from lossless_entropy_coding_amd.ffn import _LinearArgs
    a = _LinearArgs()
    base = dict(m=4, n=8, k=16, dtype=1, out_dtype=1, x=0x10000, x_stride=16, w=0x20000, w_stride=16, y=0x30000, y_stride=8,
                dy=0x40000, dy_stride=8, dx=0x50000, dx_stride=16, dw=0x60000, dw_stride=16)
    base.update(kw)
    for key, v in base.items():
        setattr(a, key, v)
    return a


@pytest.mark.parametrize("bad", [
    dict(x=0), dict(w=0), dict(y=0), dict(x=0x10001), dict(y=0x30001), dict(x_stride=15), dict(w_stride=8), dict(y_stride=7),
    dict(m=1 << 31), dict(n=1 << 30), dict(k=1 << 40), dict(dtype=0), dict(dtype=3), dict(out_dtype=0), dict(out_dtype=4),
    dict(act=4), dict(bias=0x1000, bias_dtype=2), dict(bias=0x1002, bias_dtype=3), dict(residual=0x1000, residual_stride=8),
    dict(preact=0x1000, preact_stride=15), dict(preact=0x1001, preact_stride=16), dict(x_scale=0x1000, x_scales=3),
    dict(w_scale=0x1000, w_scales=8), dict(w_scale=0x1002, w_scales=1), dict(out_scale=0x1000), dict(groups=2),
    dict(groups=5000, offsets=0x1000, w_group_stride=256), dict(groups=2, offsets=0x1000, w_group_stride=255),
    dict(workspace=0x1008), dict(status=0x1002),
], ids=str)
def test_gated_forward_refuses(ec, bad):
    assert ec.lib().gated_linear_forward(ctypes.byref(_gated(**bad)), None) == INVAL
    assert ec.lib().gated_linear_workspace_bytes(ctypes.byref(_gated(**bad))) == 0


@pytest.mark.parametrize("bad", [
    dict(dy=0), dict(preact=0), dict(preact_stride=15), dict(w=0), dict(x=0), dict(dtype=2), dict(out_dtype=2), dict(dx_stride=15),
    dict(dw_stride=15), dict(dy_stride=7), dict(dx=0x50001), dict(dw=0x60001), dict(db=0x1002), dict(act=7), dict(groups=1),
    dict(n=1 << 30), dict(groups=2, offsets=0x1000, w_group_stride=256, dw_group_stride=255), dict(),
], ids=str)
def test_gated_grad_refuses(ec, bad):
    """The last: no workspace."""
    args = _gated(**{**dict(preact=0x70000, preact_stride=16), **bad})
    assert ec.lib().gated_linear_grad(ctypes.byref(args), None) == INVAL


def test_gated_grad_workspace(ec):
    a = _gated(preact=0x70000, preact_stride=16)
    need = ec.lib().gated_linear_grad_workspace_bytes(ctypes.byref(a))
    assert need >= 4 * 16 * 2
    a.workspace, a.workspace_bytes = 0x80000, need - 1
    assert ec.lib().gated_linear_grad(ctypes.byref(a), None) == INVAL
    # rows that no tile of the input's gradient reaches
    a = _gated(preact=0x70000, preact_stride=1 << 25, n=1 << 24, dy_stride=1 << 24)
    assert ec.lib().gated_linear_grad(ctypes.byref(a), None) == UNSUPPORTED
    # sums of more columns than a launch has threads for
    a = _gated(preact=0x70000, preact_stride=1 << 29, n=1 << 28, dy_stride=1 << 28, dx=0, dw=0, db=0x1000)
    assert ec.lib().gated_linear_grad(ctypes.byref(a), None) == UNSUPPORTED


def _loss(**kw):
    from lossless_entropy_coding_amd.training import _LossArgs
    a = _LossArgs()
    base = dict(m=4, n=8, k=16, x=0x10000, x_stride=16, w=0x20000, w_stride=16, target=0x30000, target_bytes=8, dlosses=1,
                ignore_index=-100, loss=0x40000, lse=0x50000, dloss=0x60000, dx=0x70000, dx_stride=16, dw=0x80000, dw_stride=16,
                dw_dtype=1)
    base.update(kw)
    for key, v in base.items():
        setattr(a, key, v)
    return a


BAD_LOSS = [
    dict(m=1 << 31), dict(n=0), dict(n=1 << 31), dict(k=1 << 31), dict(x=0), dict(x=0x10001), dict(x_stride=15), dict(w=0),
    dict(w_stride=15), dict(target=0), dict(target=0x30004), dict(target_bytes=2), dict(target_bytes=0), dict(lse=0x50002),
    dict(status=0x1001), dict(workspace=0x1008),
]


@pytest.mark.parametrize("bad", BAD_LOSS + [dict(loss=0), dict(loss=0x40001), dict()], ids=str)
def test_loss_refuses(ec, bad):
    """The last: no workspace."""
    assert ec.lib().linear_cross_entropy(ctypes.byref(_loss(**bad)), None) == INVAL


@pytest.mark.parametrize("bad", BAD_LOSS + [
    dict(lse=0), dict(dloss=0), dict(dloss=0x60001), dict(dlosses=0), dict(dlosses=3), dict(dx=0x70001), dict(dx_stride=15),
    dict(dw=0x80001), dict(dw_stride=15), dict(dw_dtype=2), dict(dw_dtype=0), dict()], ids=str)
def test_loss_grad_refuses(ec, bad):
    assert ec.lib().linear_cross_entropy_grad(ctypes.byref(_loss(**bad)), None) == INVAL


def test_loss_workspaces(ec):
    need = ec.lib().linear_cross_entropy_grad_workspace_bytes(ctypes.byref(_loss()))
    assert need > 0
    a = _loss(workspace=0x1000000, workspace_bytes=need - 1)
    assert ec.lib().linear_cross_entropy_grad(ctypes.byref(a), None) == INVAL
    need = ec.lib().linear_cross_entropy_workspace_bytes(ctypes.byref(_loss()))
    a = _loss(workspace=0x1000000, workspace_bytes=need - 1)
    assert ec.lib().linear_cross_entropy(ctypes.byref(a), None) == INVAL
    assert ec.lib().linear_cross_entropy(ctypes.byref(_loss(m=1 << 24, workspace=0x1000000)), None) == UNSUPPORTED
    assert ec.lib().linear_cross_entropy_grad(ctypes.byref(_loss(m=1 << 26)), None) == UNSUPPORTED
    long = dict(k=1 << 28, x_stride=1 << 28, w_stride=1 << 28, dx_stride=1 << 28, dw_stride=1 << 28)
    assert ec.lib().linear_cross_entropy_grad(ctypes.byref(_loss(**long)), None) == UNSUPPORTED
    # the room for a piece of the gradient does not grow with the vocabulary
    some, more = (ec.lib().linear_cross_entropy_grad_workspace_bytes(ctypes.byref(_loss(m=4096, n=n, k=2048, x_stride=2048,
                  w_stride=2048, dx_stride=2048, dw_stride=2048))) for n in (1 << 17, 1 << 20))
    assert some == more < 1 << 30


def _adamw(count=2, **kw):
    from lossless_entropy_coding_amd.training import _AdamWArgs, _AdamWTensor
    ts = (_AdamWTensor * count)()
    for i, t in enumerate(ts):
        t.param, t.grad, t.n, t.grad_dtype = 0x10000 * (i + 1), 0x100000 * (i + 1), 300, 1
    a = _AdamWArgs()
    base = dict(m=0x1000000, v=0x2000000, m_scale=0x3000000, v_scale=0x4000000, state_blocks=2 * count, steps=0x5000000, lr=0.1,
                beta1=0.9, beta2=0.99, eps=1e-8, state_dtype=2)
    for key, v in {**base, **kw}.items():
        if key.startswith("t_"):
            setattr(ts[1], key[2:], v)
        else:
            setattr(a, key, v)
    return ts, a


@pytest.mark.parametrize("bad", [
    dict(t_param=0), dict(t_param=0x10002), dict(t_grad=0), dict(t_grad=0x100001), dict(t_grad=0x100002, t_grad_dtype=3),
    dict(t_grad_dtype=2), dict(t_grad_dtype=0), dict(t_copy=0x1001), dict(t_n=(1 << 40) + 1), dict(t_n=600), dict(state_blocks=3),
    dict(m=0), dict(v=0), dict(m=0x1000008), dict(m_scale=0), dict(v_scale=0), dict(v_scale=0x4000002), dict(steps=0),
    dict(steps=0x5000002), dict(state_dtype=1), dict(state_dtype=0), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.5),
    dict(beta2=float("nan")), dict(eps=-1e-8), dict(lr_at=0x1002), dict(grad_scale=0x1001)], ids=str)
def test_adamw_refuses(ec, bad):
    ts, a = _adamw(**bad)
    assert ec.lib().adamw_step(ts, 2, ctypes.byref(a), None) == INVAL


def test_adamw_refuses_nothing_at_all(ec):
    ts, a = _adamw()
    assert ec.lib().adamw_step(None, 2, ctypes.byref(a), None) == INVAL
    assert ec.lib().adamw_step(ts, 2, None, None) == INVAL
    assert [ec.lib().adamw_state_blocks(n) for n in (0, 1, 256, 257, 1 << 40)] == [0, 1, 1, 2, 1 << 32]


def test_binding_refuses_host_tensors(ec):
    x, w = torch.zeros(4, 16).bfloat16(), torch.zeros(16, 16).bfloat16()
    t, f = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    off = torch.tensor([0, 4], dtype=torch.int32)
    for call in [
        lambda: ec.gated_linear(x, w), lambda: ec.grouped_gated_linear(x, w[None], off), lambda: ec.grouped_gated_linear(x, w[None], None),
        lambda: ec.gated_linear_backward(x[:, :8], x, w, x), lambda: ec.grouped_gated_linear_backward(x[:, :8], x, w[None], off, x),
        lambda: ec.grouped_gated_linear_backward(x[:, :8], x, w[None], None, x),
        lambda: ec.linear_cross_entropy(x, w, t), lambda: ec.linear_cross_entropy(x=x, w=w, target=t),
        lambda: ec.linear_cross_entropy_backward(f, x, w, t, f), lambda: ec.adamw_state([f]), lambda: ec.adamw_state([]),
        lambda: ec.adamw([f], [f], ec.AdamWState(f, f, None, None, f)), lambda: ec.adamw([], [], None),
        lambda: ec.linear_cross_entropy(None, w, t), lambda: ec.linear_cross_entropy_backward(0.1, x, w, t, f),
    ]:
        with pytest.raises(ec.ECError):
            call()


@pytest.mark.gpu
def test_binding_refuses(ec):
    dev = "cuda"
    x, w = torch.zeros(4, 16, device=dev).bfloat16(), torch.zeros(16, 16, device=dev).bfloat16()
    y, z = torch.zeros(4, 8, device=dev).bfloat16(), torch.zeros(4, 16, device=dev).bfloat16()
    t, f = torch.zeros(4, dtype=torch.int64, device=dev), torch.zeros(4, device=dev)
    off = torch.tensor([0, 4], dtype=torch.int32, device=dev)
    state = ec.adamw_state([f])
    coded = ec.adamw_state([f], torch.uint8)
    s = torch.zeros(1, device=dev)
    refused = [
        lambda: ec.gated_linear(x, w[:15]), lambda: ec.gated_linear(x[:, :15], w), lambda: ec.gated_linear(x.float(), w),
        lambda: ec.gated_linear(x, w, torch.zeros(8, device=dev)), lambda: ec.gated_linear(x, w, act="tanh"),
        lambda: ec.gated_linear(x, w, out=z), lambda: ec.gated_linear(x, w, out_scale=s), lambda: ec.gated_linear(x, w, preact=y),
        lambda: ec.gated_linear(x, w, w_scale=torch.zeros(8, device=dev)), lambda: ec.gated_linear(x, w, out_dtype=torch.float16),
        lambda: ec.gated_linear(x, w.view(torch.uint8)[:, :16]), lambda: ec.gated_linear(x, w, x_scale=torch.zeros(3, device=dev)),
        lambda: ec.grouped_gated_linear(x, w[None], off.long()), lambda: ec.grouped_gated_linear(x, w[None], off[:1]),
        lambda: ec.gated_linear_backward(z, x, w, z), lambda: ec.gated_linear_backward(y, x, w, y),
        lambda: ec.gated_linear_backward(y, x, w, None), lambda: ec.gated_linear_backward(y, x, w, z, dw=w.half()),
        lambda: ec.gated_linear_backward(y, x, w, z, dw_dtype=torch.float16), lambda: ec.gated_linear_backward(y, x, w, z, dx=y),
        lambda: ec.gated_linear_backward(y, x, w, z, db=torch.zeros(8, device=dev)),
        lambda: ec.linear_cross_entropy(x, w[:0], t), lambda: ec.linear_cross_entropy(x, w, t.float()),
        lambda: ec.linear_cross_entropy(x, w, t[:3]), lambda: ec.linear_cross_entropy(x, w, t.to(torch.int16)),
        lambda: ec.linear_cross_entropy(x, w, t, ignore_index=None), lambda: ec.linear_cross_entropy(x, w, t, ignore_index=1 << 63),
        lambda: ec.linear_cross_entropy(x, w, t, loss=f.bfloat16()), lambda: ec.linear_cross_entropy(x, w, t, status=f),
        lambda: ec.linear_cross_entropy_backward(f[:3], x, w, t, f), lambda: ec.linear_cross_entropy_backward(f, x, w, t, None),
        lambda: ec.linear_cross_entropy_backward(f, x, w, t, f, dw=w[:8]),
        lambda: ec.linear_cross_entropy_backward(f, x, w, t, f, dw_dtype=torch.uint8),
        lambda: ec.adamw_state([x]), lambda: ec.adamw_state([f], torch.bfloat16), lambda: ec.adamw_state(f),
        lambda: ec.adamw([f], [f, f], state), lambda: ec.adamw([f], [f[:3]], state), lambda: ec.adamw([f], [f.half()], state),
        lambda: ec.adamw([f, f], [f, f], state), lambda: ec.adamw([f], [f], state, copies=[f]),
        lambda: ec.adamw([f], [f], state, copies=[]), lambda: ec.adamw([f], [f], state, betas=(0.9, 1.0)),
        lambda: ec.adamw([f], [f], state, eps=-1.0), lambda: ec.adamw([f], [f], state, lr=float("nan")),
        lambda: ec.adamw([f], [f], state, lr=torch.zeros(1)), lambda: ec.adamw([f], [f], state, weight_decay=[0.1, 0.1]),
        lambda: ec.adamw([f], [f], state, weight_decay=-0.1), lambda: ec.adamw([f], [f], state, seed=-1),
        lambda: ec.adamw([f], [f], state, seed=1 << 32), lambda: ec.adamw([f], [f], state, grad_scale=f),
        lambda: ec.adamw([f], [f], coded._replace(m_scale=None)), lambda: ec.adamw([f], [f], state._replace(v=coded.v)),
        lambda: ec.adamw([f], [f], state._replace(steps=s)), lambda: ec.adamw([f], [f], state._replace(m=state.m[:100])),
        lambda: ec.adamw([f[::2]], [f[:2]], state), lambda: ec.adamw([f], None, state), lambda: ec.adamw([f], [f], None),
        lambda: ec.adamw([f], [f], state[:3]), lambda: ec.adamw([f], [f], state, betas=0.9), lambda: ec.adamw([f], [f], state, lr=1e39),
    ]
    for k, call in enumerate(refused):
        with pytest.raises(ec.ECError):
            call()
            print("not refused: %d" % k)

    class Elsewhere:
        device = torch.device("cuda", torch.cuda.current_device() + 1)
        cuda_stream = 0

    for call in [lambda: ec.gated_linear(x, w, stream=Elsewhere), lambda: ec.linear_cross_entropy(x, w, t, stream=Elsewhere),
                 lambda: ec.linear_cross_entropy_backward(f, x, w, t, f, stream=Elsewhere),
                 lambda: ec.adamw([f], [f], state, stream=Elsewhere), lambda: ec.gated_linear_backward(y, x, w, z, stream=Elsewhere)]:
        with pytest.raises(ec.ECError, match="stream"):
            call()
    for call in (lambda: ec.gated_linear(x.clone().requires_grad_(), w), lambda: ec.linear_cross_entropy(x, w.clone().requires_grad_(), t)):
        with pytest.warns(UserWarning, match="autograd"):
            call()
