"""How many values a step of AdamW takes: refused by the host before anything is launched."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

from test_training_refusals import INVAL, UNSUPPORTED, _adamw, ec  # noqa: E402, F401  (ec: a fixture)


@pytest.mark.parametrize("state", [2, 3])
@pytest.mark.parametrize("sizes", [[1 << 40, 1], [1 << 39] * 3, [1] * 300 + [1 << 40], [1 << 40] * 3000], ids=lambda s: "%d tensors" % len(s))
def test_more_blocks_than_are_counted(ec, sizes, state):  # noqa: F811
    """Each tensor is within the limit of one; their blocks together are not."""
    ts, a = _adamw(len(sizes), state_blocks=(1 << 63) - 1, state_dtype=state)
    for t, n in zip(ts, sizes):
        t.n = n
    assert ec.lib().adamw_step(ts, len(sizes), ctypes.byref(a), None) == UNSUPPORTED


def test_one_tensor_has_its_own_limit(ec):  # noqa: F811
    ts, a = _adamw(1, state_blocks=(1 << 63) - 1)
    ts[0].n = (1 << 40) + 1
    assert ec.lib().adamw_step(ts, 1, ctypes.byref(a), None) == INVAL
