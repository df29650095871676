"""AdamW refuses a tensor that is listed twice, which two parts of the launch would write."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_tied_weights_are_refused():
    import lossless_entropy_coding_amd as ec
    a, b = torch.ones(300, device="cuda"), torch.ones(300, device="cuda")
    g = torch.ones(300, device="cuda").bfloat16()
    c, d = torch.zeros(300, device="cuda").bfloat16(), torch.zeros(300, device="cuda").bfloat16()
    state = ec.adamw_state([a, b])
    for params, copies in [([a, a], None), ([a, a.view(10, 30)], None), ([a, a], [c, d]), ([a, b], [c, c])]:
        with pytest.raises(ec.ECError, match="twice"):
            ec.adamw(params, [g, g], state, copies=copies)
    assert int(state.steps) == 0 and bool((a == 1).all()) and bool((c == 0).all())
    # one gradient for two tensors is only read; empty tensors and missing copies are no repetition
    e, f = torch.ones(0, device="cuda"), torch.ones(0, device="cuda")
    more = ec.adamw_state([a, e, b, f])
    ec.adamw([a, e, b, f], [g, e, g, f], more)
    ec.adamw([a, e, b, f], [g, e, g, f], more, copies=[None, None, c, None])
    assert int(more.steps) == 2 and torch.equal(a, b) and torch.equal(c, b.bfloat16())
