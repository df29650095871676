"""The C entry points with factors of a single row, whose stride may hold
anything (0 in arguments that were only zero-initialised)."""

import ctypes

import pytest

import _ffn as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ec():
    import lossless_entropy_coding_amd as ec
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ec.lib()
    return ec


def _run(ec, name, op, **kw):
    from lossless_entropy_coding_amd.ffn import _LinearArgs
    a = _LinearArgs()
    keep = []
    for key, v in kw.items():
        if isinstance(v, torch.Tensor):
            keep.append(v)
            v = v.data_ptr()
        setattr(a, key, v)
    need = ec.lib().linear_workspace_bytes(ctypes.byref(a), op)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    a.workspace, a.workspace_bytes = ws.data_ptr(), need
    assert getattr(ec.lib(), name)(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("stride", [0, 8, 64])
@pytest.mark.parametrize("n,k", [(72, 200), (64, 64), (300, 513), (1024, 1024)])
def test_one_row(ec, n, k, stride):
    """One token: its gradient of the weights, sums and inputs, and its product."""
    print("one row %d %d stride %d" % (n, k, stride), flush=True)
    g = torch.Generator(device="cuda").manual_seed(n)
    dy, x, w = _randn(g, 1, n), _randn(g, 1, k), _randn(g, n, k)
    dw, db = torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    _run(ec, "linear_grad_weight", 2, m=1, n=n, k=k, dtype=1, out_dtype=3, dy=dy, dy_stride=stride, x=x, x_stride=stride,
         dw=dw, dw_stride=k, db=db)
    R.near(dw, *R.grad_weight(dy, x, torch.float32), "dw")
    R.near(db, *R.column_sum(dy), "db")
    dx = torch.empty(1, k, dtype=torch.bfloat16, device="cuda")
    _run(ec, "linear_grad_input", 1, m=1, n=n, k=k, dtype=1, dy=dy, dy_stride=stride, w=w, w_stride=k, dx=dx, dx_stride=k)
    R.near(dx, *R.grad_input(dy, w), "dx")
    y = torch.empty(1, n, dtype=torch.bfloat16, device="cuda")
    _run(ec, "linear_forward", 0, m=1, n=n, k=k, dtype=1, out_dtype=1, x=x, x_stride=stride, w=w, w_stride=k, y=y, y_stride=n)
    want, tol, _, _ = R.linear(x, w)
    R.near(y, want, tol, "y")


@pytest.mark.parametrize("stride", [0, 8, 64])
@pytest.mark.parametrize("m,k", [(70, 200), (3, 64), (300, 513)])
def test_one_row_of_weights(ec, m, k, stride):
    """One output column; its weights hold an infinity, which no row past them may bring into the sums."""
    print("one row of weights %d %d stride %d" % (m, k, stride), flush=True)
    g = torch.Generator(device="cuda").manual_seed(m)
    dy, x, w = _randn(g, m, 1).abs() + 1, _randn(g, m, k), _randn(g, 1, k)
    y, dx = torch.empty(m, 1, dtype=torch.bfloat16, device="cuda"), torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
    _run(ec, "linear_forward", 0, m=m, n=1, k=k, dtype=1, out_dtype=1, x=x, x_stride=k, w=w, w_stride=stride, y=y, y_stride=1)
    want, tol, _, _ = R.linear(x, w)
    R.near(y, want, tol, "y")
    w[0, 5] = float("inf")
    _run(ec, "linear_grad_input", 1, m=m, n=1, k=k, dtype=1, dy=dy, dy_stride=1, w=w, w_stride=stride, dx=dx, dx_stride=k)
    assert (dx[:, 5] == float("inf")).all()
    keep = [c for c in range(k) if c != 5]
    R.near(dx[:, keep], *R.grad_input(dy, w[:, keep]), "dx")
