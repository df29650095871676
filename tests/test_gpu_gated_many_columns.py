"""The gated block on one to four rows with so many columns that a workgroup of
512 threads for every 16 of them would be more threads than a launch has."""

import pytest

torch = pytest.importorskip("torch")

import _training as tr  # noqa: E402
from _ffn import F8, near  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,kind", [(1, (1 << 27) - 16, "bf16"), (1, 1 << 27, "bf16"), (3, (1 << 27) + 40, "bf16"), (2, 1 << 27, "e4m3")])
def test_many_columns(m, n, kind):
    """2^23 workgroups of 512 threads are 2^32, which a launch takes for none."""
    import lossless_entropy_coding_amd as ec
    print("many columns %d %d %s" % (m, n, kind), flush=True)
    g = torch.Generator(device="cuda").manual_seed(m)
    k = 8 if kind == "bf16" else 16
    dtype = torch.bfloat16 if kind == "bf16" else F8

    def values(*shape):
        return torch.randint(-3, 4, shape, generator=g, device="cuda").to(dtype)

    x, probe = values(m, k), torch.tensor([0, 5, 1 << 20, n // 2 + 1, n - 17, n - 1], device="cuda")
    w = torch.zeros((2 * n, k), dtype=torch.uint8 if kind == "e4m3" else dtype, device="cuda").view(dtype)
    rows = torch.cat([probe, probe + n])
    picked = values(2 * probe.numel(), k)
    raw = torch.int16 if kind == "bf16" else torch.uint8
    w.view(raw)[rows] = picked.view(raw)
    out = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    ec.gated_linear(x, w, act=None, out=out)
    near(out[:, probe], *tr.gated(x, picked, None, None)[:2])
    out[:, probe] = 0
    assert int((out != 0).sum()) == 0           # every other column is written, with 0
