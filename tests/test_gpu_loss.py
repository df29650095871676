"""The cross entropy over a vocabulary, forward and backward, against its 64-bit form."""

import pytest

torch = pytest.importorskip("torch")

import _training as tr  # noqa: E402
from _ffn import inside_nan, near  # noqa: E402

pytestmark = pytest.mark.gpu

SIZES = [  # m, k, n
    (1, 1, 1), (1, 16, 2), (1, 64, 1000), (2, 33, 17), (16, 128, 4097), (17, 100, 130), (32, 2048, 999), (33, 64, 65),
    (70, 130, 333), (129, 1000, 2050), (300, 96, 5000), (513, 264, 257), (1030, 128, 1500), (1100, 2048, 300),
]


@pytest.fixture(scope="module")
def ec():
    import lossless_entropy_coding_amd as ec
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ec.lib()
    return ec


def _inputs(m, k, n, seed=0, scale=2.0, ignored=0.2, dtype=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((m, k), generator=g, device="cuda").bfloat16()
    w = (torch.randn((n, k), generator=g, device="cuda") * scale * k ** -0.5).bfloat16()
    t = torch.randint(n, (m,), generator=g, device="cuda")
    t = torch.where(torch.rand(m, generator=g, device="cuda") < ignored, torch.full_like(t, -100), t).to(dtype)
    return x, w, t, torch.randn(m, generator=g, device="cuda")


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward_and_backward(ec, size):
    x, w, t, dl = _inputs(*size, seed=sum(size))
    loss, lse = ec.linear_cross_entropy(x, w, t)
    want, tol, want_lse, tol_lse, _, _ = tr.loss(x, w, t)
    near(lse, want_lse, tol_lse, "lse")
    near(loss, want, tol, "loss")
    assert bool((loss[t == -100] == 0).all())
    dx, dw = ec.linear_cross_entropy_backward(dl, x, w, t, lse)
    (wx, tx), (ww, tw) = tr.loss_backward(dl, x, w, t)
    near(dx, wx, tx, "dx")
    near(dw, ww, tw, "dw")
    assert bool((dx[t == -100] == 0).all())
    again = ec.linear_cross_entropy_backward(dl, x, w, t, lse)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("m,k,n,piece", [(40000, 16, 9001, 6656), (8000, 24, 40001, 33536)])
def test_several_pieces(ec, m, k, n, piece):
    """A vocabulary of more than one piece (512 MiB of the logits' gradient, in whole 256 entries)."""
    x, w, t, dl = _inputs(m, k, n, 3)
    loss, lse = ec.linear_cross_entropy(x, w, t)
    dx, dw = ec.linear_cross_entropy_backward(dl, x, w, t, lse, dw_dtype=torch.float32)
    part = slice(0, None, 101)
    want, tol, want_lse, tol_lse, _, _ = tr.loss(x[part], w, t[part])
    near(loss[part], want, tol, "loss")
    near(lse[part], want_lse, tol_lse, "lse")
    (wx, tx), _ = tr.loss_backward(dl[part], x[part], w, t[part])
    near(dx[part], wx, tx, "dx")
    # every row's share in dw, for some entries of each piece
    sel = torch.tensor([0, 1, 4095, piece - 1, piece, piece + 255, n - 1], device="cuda")
    l = tr.mm(x.double(), w[sel].double())
    G = torch.exp(l - lse.double()[:, None])
    G -= (t[:, None] == sel[None, :]).double()
    G *= (dl.double() * (t != -100))[:, None]
    mag = tr.mm(G.abs().t().contiguous(), x.double().abs().t().contiguous())
    ww = tr.mm(G.t().contiguous(), x.double().t().contiguous())
    # G off by 2^-8 of itself, and by what lse's rounding (2^-24 of about 9) and the logits' make of it
    near(dw[sel], ww, mag * (2.0 ** -8 + 64 * tr.U) + tr.sum_error(m, mag) + tr.U * ww.abs(), "dw")


@pytest.mark.parametrize("size", [(2100, 1600, 4200), (1900, 1607, 3001), (160, 520, 16500), (256, 1536, 9000)], ids=str)
def test_large_tiles(ec, size):
    x, w, t, dl = _inputs(*size, seed=13)
    loss, lse = ec.linear_cross_entropy(x, w, t)
    want, tol, want_lse, tol_lse, _, _ = tr.loss(x, w, t)
    near(lse, want_lse, tol_lse, "lse")
    near(loss, want, tol, "loss")
    dx, dw = ec.linear_cross_entropy_backward(dl, x, w, t, lse)
    (wx, tx), (ww, tw) = tr.loss_backward(dl, x, w, t)
    near(dx, wx, tx, "dx")
    near(dw, ww, tw, "dw")


def test_targets(ec):
    x, w, t, dl = _inputs(60, 40, 100, 4)
    for other in (t.to(torch.int32), t):
        loss, lse = ec.linear_cross_entropy(x, w, other)
        assert torch.equal(loss, ec.linear_cross_entropy(x, w, t)[0])
    # another ignored value, one inside the vocabulary
    t3 = torch.where(t == -100, torch.full_like(t, 7), t)
    loss, lse = ec.linear_cross_entropy(x, w, t3, ignore_index=7)
    assert bool((loss[t3 == 7] == 0).all()) and bool((loss[t3 != 7] > 0).all())
    dx, dw = ec.linear_cross_entropy_backward(dl, x, w, t3, lse, ignore_index=7)
    (wx, tx), (ww, tw) = tr.loss_backward(dl, x, w, t3, 7)
    near(dx, wx, tx)
    near(dw, ww, tw)
    # targets outside count as ignored and are reported
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ec.linear_cross_entropy(x, w, t, status=status)
    ec.linear_cross_entropy_backward(dl, x, w, t, lse, status=status)
    assert int(status) == 0
    for bad in (100, -1, 1 << 40, -(1 << 63)):
        t4 = t.clone()
        t4[3] = bad
        t5 = t.clone()
        t5[3] = -100
        status.zero_()
        loss, lse = ec.linear_cross_entropy(x, w, t4, status=status)
        assert int(status) == ec.S_BAD_TARGET and torch.equal(loss, ec.linear_cross_entropy(x, w, t5)[0])
        status.zero_()
        got = ec.linear_cross_entropy_backward(dl, x, w, t4, lse, status=status)
        assert int(status) == ec.S_BAD_TARGET
        for a, b in zip(got, ec.linear_cross_entropy_backward(dl, x, w, t5, lse)):
            assert torch.equal(a, b)
        ec.linear_cross_entropy(x, w, t4)       # nobody asks


@pytest.mark.parametrize("m", [5, 200])
def test_no_targets(ec, m):
    """Every row ignored: no loss and no gradient, whatever the rows hold."""
    x, w, t, dl = _inputs(m, 48, 300, 5)
    t.fill_(-100)
    x[1] = float("nan")
    x[2] = float("inf")
    loss, lse = ec.linear_cross_entropy(x, w, t)
    assert bool((loss == 0).all())
    dx, dw = ec.linear_cross_entropy_backward(dl, x, w, t, lse)
    assert bool((dx == 0).all()) and bool((dw == 0).all())


@pytest.mark.parametrize("m", [6, 90, 700])
def test_masked_rows_hold_anything(ec, m):
    x, w, t, dl = _inputs(m, 64, 500, 6)
    t[0] = 5
    mask = torch.zeros(m, dtype=torch.bool, device="cuda")
    mask[1::3] = True
    t = torch.where(mask, torch.full_like(t, -100), t)
    clean = x.clone()
    x[1] = float("nan")
    x[4] = float("-inf")
    lse = ec.linear_cross_entropy(x, w, t)[1]
    loss, clean_lse = ec.linear_cross_entropy(clean, w, t)
    assert torch.equal(ec.linear_cross_entropy(x, w, t)[0], loss)
    dl[1] = float("nan")
    for a, b in zip(ec.linear_cross_entropy_backward(dl, x, w, t, lse),
                    ec.linear_cross_entropy_backward(dl.nan_to_num(), clean, w, t, clean_lse)):
        assert torch.equal(a, b)


def test_far_logits(ec):
    """Logits of thousands: the maximum is taken out before the exponentials; one entry has all the probability."""
    m, k, n = 70, 64, 1000
    x, w, t, dl = _inputs(m, k, n, 7, scale=400.0)
    t[: m // 2] = tr.mm(x.double(), w.double()).argmax(1)[: m // 2]
    loss, lse = ec.linear_cross_entropy(x, w, t)
    want, tol, want_lse, tol_lse, _, _ = tr.loss(x, w, t)
    assert float(want.max()) > 1000
    near(loss, want, tol)
    near(lse, want_lse, tol_lse)
    assert bool(loss.isfinite().all()) and bool((loss >= 0).all())


def test_vocabulary_entries_of_minus_infinity(ec):
    """Logits of -inf (entries that are switched off) have no probability, in whole tiles too."""
    m, k, n = 40, 16, 700
    x, w, t, dl = _inputs(m, k, n, 8, ignored=0)
    x[:, 0] = 1.0
    w[:, 0] = 0.0
    for rows in (4, 40):
        for cut in (300, 512):
            a, b, s = x[:rows].contiguous(), w.clone(), (t % cut)[:rows].contiguous()
            b[cut:] = 0.0
            b[cut:, 0] = float("-inf")
            loss, lse = ec.linear_cross_entropy(a, b, s)
            want, tol, want_lse, tol_lse, _, _ = tr.loss(a, w[:cut], s)
            near(loss, want, tol)
            near(lse, want_lse, tol_lse)


@pytest.mark.parametrize("m", [3, 200])
def test_special_values_stay_in_their_row(ec, m):
    x, w, t, dl = _inputs(m, 64, 500, 9, ignored=0)
    clean = ec.linear_cross_entropy(x, w, t)
    x[1, 2] = float("nan")
    loss, lse = ec.linear_cross_entropy(x, w, t)
    rows = [i for i in range(m) if i != 1]
    assert torch.equal(loss[rows], clean[0][rows]) and torch.equal(lse[rows], clean[1][rows])
    assert bool(loss[1].isnan()) and bool(lse[1].isnan())


def test_strides_and_buffers(ec):
    for m, k, n in [(5, 65, 77), (80, 71, 300), (90, 64, 130)]:
        x, w, t, dl = _inputs(m, k, n, 10)
        loss, lse = ec.linear_cross_entropy(x, w, t)
        out, out_lse = torch.empty_like(loss), torch.empty_like(lse)
        got = ec.linear_cross_entropy(inside_nan(x), inside_nan(w, left=1), t, loss=out, lse=out_lse)
        assert got[0] is out and got[1] is out_lse
        near(out, *tr.loss(x, w, t)[:2])
        dx = inside_nan(torch.zeros(m, k, device="cuda").bfloat16())
        dw = inside_nan(torch.zeros(n, k, device="cuda"), left=1)
        ec.linear_cross_entropy_backward(dl, inside_nan(x), inside_nan(w, left=1), t, lse, dx=dx, dw=dw)
        (wx, tx), (ww, tw) = tr.loss_backward(dl, x, w, t, dw_dtype=torch.float32)
        near(dx, wx, tx)
        near(dw, ww, tw)
        for base, (rows, cols), left in ((dx._base, (m, k), 3), (dw._base, (n, k), 1)):
            keep = torch.ones_like(base, dtype=torch.bool)
            keep[2:2 + rows, left:left + cols] = False
            assert bool(base[keep].isnan().all())
        one = ec.linear_cross_entropy_backward(dl, x, w, t, lse, need_dw=False)
        two = ec.linear_cross_entropy_backward(dl, x, w, t, lse, need_dx=False, dw_dtype=torch.float32)
        assert one[1] is None and two[0] is None
        near(one[0], wx, tx)
        near(two[1], ww, tw)
        # one gradient for all rows
        same = torch.full((1,), 0.25, device="cuda")
        for a, b in zip(ec.linear_cross_entropy_backward(same, x, w, t, lse),
                        ec.linear_cross_entropy_backward(same.expand(m).contiguous(), x, w, t, lse)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("m,k,n", [(0, 16, 8), (5, 0, 8), (0, 0, 1)])
def test_empty(ec, m, k, n):
    x, w = torch.zeros(m, k, device="cuda").bfloat16(), torch.ones(n, k, device="cuda").bfloat16()
    t = torch.zeros(m, dtype=torch.int64, device="cuda")
    loss, lse = ec.linear_cross_entropy(x, w, t)
    assert loss.shape == (m,) and torch.allclose(loss.double(), torch.full((m,), float(n), device="cuda").double().log())
    dx, dw = ec.linear_cross_entropy_backward(torch.ones(m, device="cuda") if m else torch.ones(1, device="cuda"), x, w, t, lse)
    assert dx.shape == x.shape and dw.shape == w.shape and bool((dw == 0).all())


def test_by_differences(ec):
    m, k, n = 9, 24, 50
    x, w, t, dl = _inputs(m, k, n, 11)
    lse = ec.linear_cross_entropy(x, w, t)[1]
    dx, dw = ec.linear_cross_entropy_backward(dl, x, w, t, lse, dw_dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(1)
    kept = t != -100

    def value(x, w):
        l = tr.mm(x, w)
        each = torch.logsumexp(l, 1) - l[torch.arange(m, device="cuda"), t.clamp(min=0)]
        return float((each * dl.double() * kept).sum())

    for which, grad in (("x", dx), ("w", dw)):
        v = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        args = {"x": x.double(), "w": w.double()}
        plus, minus = dict(args), dict(args)
        plus[which], minus[which] = args[which] + 1e-4 * v, args[which] - 1e-4 * v
        slope = (value(**plus) - value(**minus)) / 2e-4
        # G and dx are rounded to bf16
        (wx, tx), (ww, tw) = tr.loss_backward(dl, x, w, t, dw_dtype=torch.float32)
        room = float(((tx if which == "x" else tw) * v.abs()).sum()) + 1e-6 * abs(slope)
        assert abs(slope - float((grad.double() * v).sum())) <= room


def test_stream_and_graph(ec):
    x, w, t, dl = _inputs(300, 72, 1500, 12)
    side = torch.cuda.Stream()

    def both():
        loss, lse = ec.linear_cross_entropy(x, w, t)
        return (loss, lse) + ec.linear_cross_entropy_backward(dl, x, w, t, lse)

    want = both()
    torch.cuda.synchronize()
    got = ec.linear_cross_entropy(x, w, t, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0])
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = both()
    for k in range(3):
        x2, _, t2, _ = _inputs(300, 72, 1500, 20 + k, ignored=0.3 * k)      # another number of rows with a target
        x.copy_(x2)
        t.copy_(t2)
        graph.replay()
        torch.cuda.synchronize()
        eager = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager)), "replay %d" % k
