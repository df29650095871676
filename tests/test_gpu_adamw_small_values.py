"""AdamW with e4m3 states where the gradients of one block of 256 values are far
apart: values whose v is held as 0 still move by a few lr at most."""

import pytest

torch = pytest.importorskip("torch")

import _training as tr  # noqa: E402
from _ffn import near, values  # noqa: E402

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
BLOCK = 256
B1, B2, EPS, LR = 0.9, 0.999, 1e-8, 1e-3


@pytest.fixture(scope="module")
def ec():
    import lossless_entropy_coding_amd as ec
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ec.lib()
    return ec


def _expected(p, g, m, v, least, step):
    """p after the step from values in 64 bits, v's root at least `least`, and the error of 32 bits: as in
    ``tr.adamw``, but that a root which is `least` is off by 3 u of it (two roundings and b2's root)."""
    want = tr.adamw(p, g, m, v, step, LR, (B1, B2), EPS, 0.0)
    m2, em = want["m"]
    v2, ev = want["v"]
    c1, c2 = 1 - B1 ** step, 1 - B2 ** step
    below = torch.maximum(v2.sqrt(), least) / c2 ** 0.5 + EPS
    change = LR * m2 / c1 / below
    share = torch.where(v2 > 0, ev / v2, torch.zeros_like(v2)) + 3 * tr.U
    p2 = p - change
    return p2, change.abs() * (24 * tr.U + share) + LR / c1 * em / below + tr.U * (4 * p.abs() + 2 * p2.abs())


@pytest.mark.parametrize("largest", [1.0, 0.01])
@pytest.mark.parametrize("ratio", [1e-4, 1e-5, 1e-6, 1e-7])
def test_change_is_bounded(ec, ratio, largest):
    """One value in 256 has gradients of size `largest`, the others `ratio` times that.  Each step is the formula's, and
    after 20 steps none moves a small value by more than 8 lr.  (Exact states: at most (1 - b1) / sqrt((1 - b2) (1 - b1^2
    / b2)) = 7.3 lr, by the Cauchy-Schwarz inequality on the two sums.  m held as one step while its value is less
    than that adds the ratio of the two scales, here below 1, over the share that b2 leaves.)"""
    n = 10 * BLOCK
    gen = torch.Generator(device="cuda").manual_seed(5)
    size = torch.full((n,), largest * ratio, device="cuda")
    size[::BLOCK] = largest
    small = torch.ones(n, dtype=torch.bool, device="cuda")
    small[::BLOCK] = False
    p = torch.zeros(n, device="cuda")
    state = ec.adamw_state([p], F8)
    held_as_zero = 0
    for step in range(1, 301):
        g = torch.randn(n, generator=gen, device="cuda") * size
        m, v = tr.held(state, "m"), tr.held(state, "v")
        least = B2 ** 0.5 * 2.0 ** -9 * state.v_scale.double().repeat_interleave(BLOCK)
        before = p.double()
        held_as_zero += int(((v == 0) & (m != 0) & small).sum())
        ec.adamw([p], [g], state, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=0.0, seed=11)
        near(p, *_expected(before, g.double(), m, v, least, step), "step %d" % step)
        if step > 20:
            moved = float((p.double() - before).abs()[small].max()) / LR
            assert moved <= 8, "step %d moved a value by %g lr" % (step, moved)
    assert ratio > 1e-5 or held_as_zero > 100           # the case is met


def test_not_finite_stays(ec):
    """A v that was not finite is NaN, not the least: p becomes NaN too, whatever m is."""
    p = torch.zeros(300, device="cuda")
    g = torch.full((300,), 0.01, device="cuda")
    g[7] = 1e20                                 # its square is infinite, m is not
    state = ec.adamw_state([p], F8)
    ec.adamw([p], [g], state)
    assert bool(values(state.v)[7].isnan()) and bool(values(state.m)[7].isfinite())
    g[7] = 0.01
    ec.adamw([p], [g], state)
    rest = torch.ones(300, dtype=torch.bool, device="cuda")
    rest[7] = False
    assert bool(p[7].isnan()) and bool(p[rest].isfinite().all())
