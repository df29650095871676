"""Rows longer than a tile's 32-bit offsets reach: what a plan copies (on the
CPU, from the workspace it asks for), what is refused, and sums over long
contractions against 64-bit forms.

In the GPU tests one factor is zero outside a few windows of the contraction,
so a sum has as many terms as the windows hold: zeros add nothing to it, and
the tolerance is that of the windows' length."""

import ctypes

import pytest

import _ffn as R

torch = pytest.importorskip("torch")

F8 = R.F8
FORWARD, GRAD_INPUT, GRAD_WEIGHT = 0, 1, 2
OK, UNSUPPORTED = 0, 2
MIB = 1 << 20


@pytest.fixture(scope="module")
def ec():
    import os
    import lossless_entropy_coding_amd as ec
    if not os.path.exists(ec.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    ec.lib()
    return ec


def _args(m, n, k, dtype=1, **kw):
    """Aligned arguments of packed rows (the pointers are never read by the host)."""
    from lossless_entropy_coding_amd.ffn import _LinearArgs
    a = _LinearArgs()
    base = dict(m=m, n=n, k=k, dtype=dtype, out_dtype=1, x=0x10000, x_stride=k, w=0x20000, w_stride=k, y=0x30000, y_stride=n,
                dy=0x40000, dy_stride=n, dx=0x50000, dx_stride=k, dw=0x60000, dw_stride=k)
    base.update(kw)
    for key, v in base.items():
        setattr(a, key, v)
    return a


def _workspace(ec, a, op):
    return ec.lib().linear_workspace_bytes(ctypes.byref(a), op)


@pytest.mark.parametrize("m,n,k,dtype", [(64, 64, 17_300_480, 1), (512, 1024, 4_500_480, 1), (1024, 1024, 4_300_000, 1),
                                         (64, 64, 34_000_000, 2), (300, 70, 1 << 30, 2), (33, 8, (1 << 31) - 16, 2)])
def test_long_rows_are_not_copied(ec, m, n, k, dtype):
    """A copy of packed rows reaches no further than the rows do; what a plan may ask for are partial sums, of at most
    32 splits of whole tiles."""
    tiles = (m + 255) // 256 * ((n + 255) // 256) * 65536
    assert _workspace(ec, _args(m, n, k, dtype), FORWARD) <= 32 * tiles * 4


def test_strides_within_reach_are_read_in_place(ec):
    a = _args(512, 512, 512, x_stride=1 << 22, w_stride=1 << 22)     # 8 MiB a row, 512 rows: read in place by tiles of 128
    assert _workspace(ec, a, FORWARD) in (0,) + tuple(s * 512 * 512 * 4 for s in (2, 4, 8, 16, 32))
    a = _args(512, 512, 512, dy_stride=1 << 24, x_stride=1 << 24)     # 32 rows of 32 MiB
    assert _workspace(ec, a, GRAD_WEIGHT) in tuple(s * 512 * 512 * 4 for s in (0, 2, 4, 8, 16, 32))


@pytest.mark.parametrize("op,m,n,k", [(GRAD_INPUT, 64, 1 << 24, 8), (GRAD_INPUT, 64, 8, 1 << 25), (GRAD_WEIGHT, 64, 1 << 25, 8),
                                      (GRAD_WEIGHT, 64, 8, 1 << 25), (GRAD_INPUT, 64, 1 << 30, 1 << 10)])
def test_backward_refuses_longer_rows(ec, op, m, n, k):
    f = ec.lib().linear_grad_input if op == GRAD_INPUT else ec.lib().linear_grad_weight
    a = _args(m, n, k)
    assert _workspace(ec, a, op) == 0
    assert f(ctypes.byref(a), None) == UNSUPPORTED
    a.db = 0x70000                                  # nothing is launched for the other result either
    assert f(ctypes.byref(a), None) == UNSUPPORTED


def test_longest_rows_of_the_backward_products_fit(ec):
    for op, n, k in [(GRAD_INPUT, (1 << 24) - 1024, 8), (GRAD_INPUT, 8, (1 << 25) - 2048),
                     (GRAD_WEIGHT, (1 << 25) - 2048, 8), (GRAD_WEIGHT, 8, (1 << 25) - 2048)]:
        a = _args(64, n, k)
        inside = _workspace(ec, a, op)
        assert inside <= 32 * 64 * 64 * 4           # at most the partial sums of one tile's splits
        a.dy, a.x, a.w = a.dy + 2, a.x + 2, a.w + 2
        assert _workspace(ec, a, op) > inside + 15 * max(n, k)


def _windows(k, width):
    """Starts of windows at both ends and at the places where 32-bit offsets of bf16 or e4m3 rows end."""
    at = {0, k - width, k // 2 - width // 2}
    for edge in (1 << 22, 1 << 23, 1 << 24, 1 << 25):
        if edge + width < k:
            at.add(edge - width // 2)
    return sorted(at)


def _fill(g, t, scale, lo, hi):
    """Random values in columns lo .. hi - 1."""
    v = torch.randn(t.shape[0], hi - lo, generator=g, device="cuda") * scale
    t[:, lo:hi] = v.clamp(-448, 448).to(t.dtype) if t.dtype == F8 else v.to(t.dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k,kind", [(64, 64, 17_300_480, torch.bfloat16), (130, 300, 4_500_480, torch.bfloat16),
                                        (260, 257, 4_300_000, torch.bfloat16), (40, 70, 34_000_016, F8),
                                        (33, 40, 17_300_003, torch.bfloat16), (300, 40, 9_000_000, F8)])
def test_long_contraction(ec, m, n, k, kind):
    print("long rows %d %d %d %s" % (m, n, k, kind), flush=True)
    g = torch.Generator(device="cuda").manual_seed(m)
    width = 64
    at = _windows(k, width)
    x, w = torch.empty(m, k, dtype=kind, device="cuda"), torch.zeros(n, k, dtype=kind, device="cuda")
    for lo in range(0, k, 1 << 20):
        _fill(g, x, 1.0, lo, min(k, lo + (1 << 20)))
    for lo in at:
        _fill(g, w, 1.0, lo, lo + width)
    cols = torch.cat([torch.arange(lo, lo + width, device="cuda") for lo in at])
    x0, w0 = (t.view(torch.uint8)[:, cols].view(F8) if kind == F8 else t[:, cols] for t in (x, w))
    want, tol, _, _ = R.linear(x0, w0, out=torch.float32)
    R.near(ec.linear(x, w, out_dtype=torch.float32), want, tol, "y")
    off = torch.tensor([0, m // 3, m], dtype=torch.int32, device="cuda")
    y = ec.grouped_linear(x, torch.stack([w, w]) if m < 100 else w[None], off if m < 100 else off[[0, 2]], out_dtype=torch.float32)
    R.near(y, want, tol, "grouped y")


@pytest.mark.gpu
def test_long_rows_of_the_backward_products(ec):
    """n and k beyond the reach of a large tile, up to the longest."""
    g = torch.Generator(device="cuda").manual_seed(3)
    m, width = 40, 64
    for n, k in [(5_000_000, 24), (24, 5_000_000), ((1 << 24) - 1024, 16), (16, (1 << 25) - 2048)]:
        print("backward of long rows %d %d" % (n, k), flush=True)
        dy, w, x = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((m, n), (n, k), (m, k)))
        if n > k:
            cols = torch.cat([torch.arange(lo, lo + width, device="cuda") for lo in _windows(n, width)])
            dy[:, cols] = torch.randn(m, len(cols), generator=g, device="cuda").bfloat16()
            w[:] = torch.randn(n, k, generator=g, device="cuda").bfloat16()
            x[:] = torch.randn(m, k, generator=g, device="cuda").bfloat16()
            dx, dw, _ = ec.linear_backward(dy, x, w, need_db=False)
            R.near(dx, *R.grad_input(dy[:, cols], w[cols]), "dx")
            R.near(dw[cols], *R.grad_weight(dy[:, cols], x), "dw")
            assert int((dw != 0).any(1).sum()) <= len(cols)
        else:
            cols = torch.cat([torch.arange(lo, lo + width, device="cuda") for lo in _windows(k, width)])
            dy[:] = torch.randn(m, n, generator=g, device="cuda").bfloat16()
            w[:, cols] = torch.randn(n, len(cols), generator=g, device="cuda").bfloat16()
            x[:, cols] = torch.randn(m, len(cols), generator=g, device="cuda").bfloat16()
            dx, dw, _ = ec.linear_backward(dy, x, w, need_db=False)
            R.near(dx[:, cols], *R.grad_input(dy, w[:, cols]), "dx")
            R.near(dw[:, cols], *R.grad_weight(dy, x[:, cols]), "dw")
            assert int((dx != 0).any(0).sum()) <= len(cols) and int((dw != 0).any(0).sum()) <= len(cols)


@pytest.mark.gpu
def test_more_than_2_30_tokens(ec):
    """The weight gradient's contraction runs over the tokens, walked to its end."""
    g = torch.Generator(device="cuda").manual_seed(4)
    m, n, k, last = (1 << 30) + 1000, 8, 16, 5000
    dy, x = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda"), torch.ones(m, k, dtype=torch.bfloat16, device="cuda")
    dy[-last:] = torch.randn(last, n, generator=g, device="cuda").bfloat16()
    x[-last:] = torch.randn(last, k, generator=g, device="cuda").bfloat16()
    _, dw, db = ec.linear_backward(dy, x, torch.empty(n, k, dtype=torch.bfloat16, device="cuda"), need_dx=False,
                                   dw_dtype=torch.float32)
    R.near(dw, *R.grad_weight(dy[-last:], x[-last:], torch.float32), "dw")
    R.near(db, *R.column_sum(dy[-last:]), "db")


def test_launches_too_large_are_refused(ec):
    """A launch has fewer than 2^32 threads: 512 for each 256 columns here."""
    f = ec.lib().linear_forward
    assert f(ctypes.byref(_args(1, (1 << 31) - 1, 8)), None) == UNSUPPORTED
    a = _args(40, 1 << 30, 40)
    a.w = a.w + 2                                   # a copy of 80 GiB
    assert f(ctypes.byref(a), None) == UNSUPPORTED and _workspace(ec, a, FORWARD) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 20])
def test_many_columns(ec, m):
    """More columns than the kernel for few rows can be launched for."""
    print("many columns %d" % m, flush=True)
    g = torch.Generator(device="cuda").manual_seed(m)
    n, k = 300_000_001, 8
    x = torch.randn(m, k, generator=g, device="cuda").bfloat16()
    w = torch.empty(n, k, dtype=torch.bfloat16, device="cuda")
    for lo in range(0, n, 1 << 24):
        hi = min(n, lo + (1 << 24))
        w[lo:hi] = torch.randn(hi - lo, k, generator=g, device="cuda").bfloat16()
    y = ec.linear(x, w)
    for lo in (0, (1 << 28) - 5000, n - 20000, n // 2):
        s = slice(lo, lo + 20000)
        want, tol, _, _ = R.linear(x, w[s])
        R.near(y[:, s], want, tol, "y from column %d" % lo)
    for lo in range(0, n, 1 << 24):                 # every column was written: by a float product, roughly
        hi = min(n, lo + (1 << 24))
        assert torch.allclose(y[:, lo:hi].float(), x.float() @ w[lo:hi].float().t().contiguous(), rtol=0.05, atol=0.05)
