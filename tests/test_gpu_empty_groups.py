"""Grouped products with nothing to compute report bad offsets all the same."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ec():
    import lossless_entropy_coding_amd as ec
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ec.lib()
    return ec


@pytest.mark.parametrize("m,n,k", [(0, 8, 16), (5, 0, 16), (5, 8, 0), (0, 0, 0), (5, 8, 16)])
@pytest.mark.parametrize("offsets", [[0, 3, 9], [0, 2, 1], [-1, 0, 0], [0, 0, 0]])
def test_status(ec, m, n, k, offsets):
    print("empty %d %d %d %s" % (m, n, k, offsets), flush=True)
    x, dy, w = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((m, k), (m, n), (2, n, k)))
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    bad = any(v < 0 or v > m for v in offsets) or offsets != sorted(offsets)
    want = ec.S_BAD_OFFSETS if bad else 0

    def status(call):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(st)
        return int(st)

    assert status(lambda st: ec.grouped_linear(x, w, off, status=st)) == want
    assert status(lambda st: ec.grouped_linear_backward(dy, x, w, off, status=st)) == want
    assert status(lambda st: ec.grouped_linear_backward(dy, x, w, off, need_dx=False, need_db=False, status=st)) == want
    assert status(lambda st: ec.grouped_linear_backward(dy, x, w, off, need_dx=False, need_dw=False, status=st)) == want
    assert status(lambda st: ec.grouped_linear_backward(dy, x, w, off, need_dw=False, need_db=False, status=st)) == want
