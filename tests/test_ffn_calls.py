"""How the feed-forward operators may be called: arguments by name, streams,
wrong kinds of objects, tensors that require gradients."""

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ec():
    import os
    import lossless_entropy_coding_amd as ec
    if not os.path.exists(ec.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    ec.lib()
    return ec


def _inputs(device):
    g = torch.Generator().manual_seed(2)

    def randn(*shape):
        return torch.randn(shape, generator=g).bfloat16().to(device)

    return dict(x=randn(5, 16), w=randn(8, 16), dy=randn(5, 8), dyn=randn(5, 16), we=randn(2, 8, 16),
                off=torch.tensor([0, 2, 5], dtype=torch.int32, device=device),
                mean=torch.zeros(5, device=device), rstd=torch.ones(5, device=device))


def _calls(ec, t):
    """(by position, by name) for each of the six."""
    return [
        (lambda: ec.linear(t["x"], t["w"]), lambda: ec.linear(w=t["w"], x=t["x"])),
        (lambda: ec.grouped_linear(t["x"], t["we"], t["off"]),
         lambda: ec.grouped_linear(offsets=t["off"], x=t["x"], w=t["we"])),
        (lambda: ec.linear_backward(t["dy"], t["x"], t["w"]), lambda: ec.linear_backward(x=t["x"], w=t["w"], dy=t["dy"])),
        (lambda: ec.grouped_linear_backward(t["dy"], t["x"], t["we"], t["off"]),
         lambda: ec.grouped_linear_backward(dy=t["dy"], x=t["x"], w=t["we"], offsets=t["off"])),
        (lambda: ec.layer_norm(t["x"]), lambda: ec.layer_norm(x=t["x"], eps=1e-5)),
        (lambda: ec.layer_norm_backward(t["dyn"], t["x"], t["mean"], t["rstd"]),
         lambda: ec.layer_norm_backward(dy=t["dyn"], x=t["x"], mean=t["mean"], rstd=t["rstd"])),
    ]


def test_names_reach_the_checks(ec):
    """On host tensors every call is refused by the operator's own checks, however its arguments are given."""
    for calls in _calls(ec, _inputs("cpu")):
        for call in calls:
            with pytest.raises(ec.ECError):
                call()
    for f in (ec.linear, ec.layer_norm, ec.linear_backward):
        with pytest.raises(TypeError):
            f()


@pytest.mark.gpu
def test_names_give_the_same(ec):
    for by_position, by_name in _calls(ec, _inputs("cuda")):
        a, b = by_position(), by_name()
        a, b = (v if isinstance(v, tuple) else (v,) for v in (a, b))
        assert len(a) == len(b) and all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.gpu
def test_stream_of_another_device_is_refused(ec):
    """Only what the binding reads of a stream: there may be no second device here to make one on."""
    class Elsewhere:
        device = torch.device("cuda", torch.cuda.current_device() + 1)
        cuda_stream = 0

    t = _inputs("cuda")
    for call in [lambda s: ec.linear(t["x"], t["w"], stream=s), lambda s: ec.layer_norm(x=t["x"], stream=s),
                 lambda s: ec.grouped_linear(t["x"], t["we"], t["off"], stream=s),
                 lambda s: ec.linear_backward(t["dy"], t["x"], t["w"], stream=s)]:
        with pytest.raises(ec.ECError, match="stream"):
            call(Elsewhere)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = ec.linear(x=t["x"], w=t["w"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, ec.linear(t["x"], t["w"]))


@pytest.mark.gpu
def test_objects_that_are_no_tensors_are_refused(ec):
    t = _inputs("cuda")
    dev = [1.0]
    bf = torch.bfloat16
    for call in [lambda: ec.linear(t["x"], t["w"], out=dev, out_dtype=bf), lambda: ec.linear(t["x"], t["w"], out=dev),
                 lambda: ec.linear(t["x"], t["w"], dev), lambda: ec.linear(t["x"], t["w"], residual=dev),
                 lambda: ec.linear(t["x"], t["w"], preact=dev), lambda: ec.linear(t["x"], t["w"], x_scale=2.0),
                 lambda: ec.grouped_linear(t["x"], t["we"], t["off"], status=0),
                 lambda: ec.grouped_linear(t["x"], t["we"], [0, 2, 5]),
                 lambda: ec.linear_backward(t["dy"], t["x"], t["w"], dw=dev),
                 lambda: ec.linear_backward(t["dy"], t["x"], t["w"], dw=dev, dw_dtype=bf),
                 lambda: ec.linear_backward(t["dy"], t["x"], t["w"], db=dev), lambda: ec.linear_backward(t["dy"], dev, t["w"]),
                 lambda: ec.linear_backward(t["dy"], t["x"], t["w"], dx=dev),
                 lambda: ec.linear_backward(t["dy"], t["x"], t["w"], preact=dev, act="gelu"),
                 lambda: ec.layer_norm(t["x"], out=dev, out_dtype=bf), lambda: ec.layer_norm(t["x"], out=dev),
                 lambda: ec.layer_norm(t["x"], mean=dev, rstd=dev), lambda: ec.layer_norm(t["x"], weight=1.0),
                 lambda: ec.layer_norm_backward(t["dyn"], t["x"], t["mean"], 1.0)]:
        with pytest.raises(ec.ECError):
            call()


@pytest.mark.gpu
def test_unrecorded_gradients_are_warned_of(ec):
    """Where torch records and a tensor requires its gradient; the values are the same, and silent otherwise."""
    import warnings
    t = _inputs("cuda")
    bias, res, norm = torch.ones(8, device="cuda"), torch.ones(5, 8, device="cuda").bfloat16(), torch.ones(16, device="cuda")
    calls = [lambda g: ec.linear(g(t["x"]), t["w"]), lambda g: ec.linear(x=t["x"], w=g(t["w"])),
             lambda g: ec.linear(t["x"], t["w"], g(bias)), lambda g: ec.linear(t["x"], t["w"], residual=g(res)),
             lambda g: ec.grouped_linear(t["x"], g(t["we"]), t["off"]), lambda g: ec.layer_norm(g(t["x"]))[0],
             lambda g: ec.layer_norm(t["x"], g(norm))[0]]
    for call in calls:
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            want = call(lambda v: v)
            with torch.no_grad():
                assert torch.equal(call(lambda v: v.clone().requires_grad_()), want)
        with pytest.warns(UserWarning, match="autograd does not record") as seen:
            got = call(lambda v: v.clone().requires_grad_())
        assert torch.equal(got, want) and not got.requires_grad
        assert len(seen) == 1 and seen[0].filename == __file__
