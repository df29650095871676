"""The cross entropy's loss where the logits are far from zero: it has its own
accuracy, not that of the log of the sum of exponentials beside it."""

import math

import pytest

torch = pytest.importorskip("torch")

from _ffn import U  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("level", [0.0, 64.0, 8192.0, -8192.0])
@pytest.mark.parametrize("m,n", [(1, 1000), (3, 4097), (70, 1000), (300, 5000), (1100, 333), (700, 20000)])
def test_equal_logits(m, n, level):
    """Every logit is `level`, exactly: the sum is n, the loss log n, off by a logarithm's error (2 steps of it)."""
    import lossless_entropy_coding_amd as ec
    x = torch.zeros((m, 16), device="cuda").bfloat16()
    x[:, 0] = 1
    w = torch.zeros((n, 16), device="cuda").bfloat16()
    w[:, 0] = level
    target = torch.arange(m, device="cuda") * 7 % n
    loss, lse = ec.linear_cross_entropy(x, w, target)
    want = math.log(n)
    assert float((loss.double() - want).abs().max()) <= 4 * U * want
    assert float((lse.double() - (level + want)).abs().max()) <= 4 * U * want + U * abs(level + want)


@pytest.mark.parametrize("m", [2, 40, 400])
def test_sure_rows(m):
    """The target's logit is 96, another one 88, the rest -100: the loss is log(1 + e^-8) = 3.4e-4, off by the rounding
    of the sum (half a step of 1, and the exponential's (3 * 8 + 4) u of e^-8) and of the logarithm, never negative; the
    row of the other one has 8 more."""
    import lossless_entropy_coding_amd as ec
    n = 3000
    x = torch.zeros((m, 16), device="cuda").bfloat16()
    x[:, 0] = 1
    w = torch.zeros((n, 16), device="cuda").bfloat16()
    w[:, 0] = -100
    w[17, 0], w[2900, 0] = 96, 88
    target = torch.full((m,), 17, device="cuda")
    target[::2] = 2900
    loss, _ = ec.linear_cross_entropy(x, w, target)
    want = math.log1p(math.exp(-8.0))
    sure = loss[1::2].double()
    if sure.numel():
        assert float((sure - want).abs().max()) <= U * (2 + 28 * math.exp(-8.0) + 4 * want) and float(sure.min()) >= 0
    assert float((loss[::2].double() - (8 + want)).abs().max()) <= U * (2 + 8 + 1)
