"""The operators of a training step together: norm, gated block, product with
the residual, loss, backward pass and weight update, in bf16 with fp32 masters,
against the same step in 64 bits, and captured into a graph."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

import _ffn  # noqa: E402
import _training as tr  # noqa: E402

pytestmark = pytest.mark.gpu

ROWS, WIDTH, HIDDEN, VOCABULARY = 96, 64, 136, 500


@pytest.fixture(scope="module")
def ec():
    import lossless_entropy_coding_amd as ec
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ec.lib()
    return ec


class Model:
    """fp32 masters and the bf16 weights that the layer works with."""

    def __init__(self, ec, state=torch.float32, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(shape, generator=g, device="cuda") * scale

        self.masters = [normal(2 * HIDDEN, WIDTH, scale=WIDTH ** -0.5), normal(WIDTH, HIDDEN, scale=HIDDEN ** -0.5),
                        normal(VOCABULARY, WIDTH, scale=WIDTH ** -0.5), 1 + normal(WIDTH, scale=0.1), normal(WIDTH, scale=0.1),
                        normal(2 * HIDDEN, scale=0.1)]
        self.weights = [p.bfloat16() for p in self.masters[:3]]
        self.state = ec.adamw_state(self.masters, state)

    def gradients(self, ec, x, target):
        w1, w2, w3 = self.weights
        _, _, _, gain, shift, b1 = self.masters
        h, mean, rstd = ec.layer_norm(x, gain, shift)
        a, z = ec.gated_linear(h, w1, b1, act="gelu", save_preact=True)
        y = ec.linear(a, w2, residual=x)
        loss, lse = ec.linear_cross_entropy(y, w3, target)
        each = torch.full((1,), 1.0 / target.numel(), device="cuda")
        dy, dw3 = ec.linear_cross_entropy_backward(each, y, w3, target, lse)
        da, dw2, _ = ec.linear_backward(dy, a, w2, need_db=False)
        dh, dw1, db1 = ec.gated_linear_backward(da, h, w1, z, act="gelu")
        dx, dgain, dshift = ec.layer_norm_backward(dh, x, mean, rstd, gain, residual_grad=dy)
        return loss, dx, [dw1, dw2, dw3, dgain, dshift, db1]

    def step(self, ec, x, target):
        loss, _, grads = self.gradients(ec, x, target)
        ec.adamw(self.masters, grads, self.state, lr=0.01, weight_decay=[0.1, 0.1, 0.1, 0, 0, 0],
                 copies=self.weights + [None] * 3)
        return loss


def _data(seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((ROWS, WIDTH), generator=g, device="cuda").bfloat16()
    t = torch.randint(VOCABULARY, (ROWS,), generator=g, device="cuda")
    t[::7] = -100
    return x, t


def _exact(model, x, target):
    """The loss's mean by rows in 64 bits, with autograd's gradients of x and of every weight."""
    leaves = [w.double().requires_grad_() for w in model.weights] + [p.double().requires_grad_() for p in model.masters[3:]]
    w1, w2, w3, gain, shift, b1 = leaves
    x = x.double().requires_grad_()
    centred = x - x.mean(1, keepdim=True)
    h = centred / (centred.square().mean(1, keepdim=True) + 1e-5).sqrt() * gain + shift
    z = h @ w1.t() + b1
    y = (tr.act(z[:, :HIDDEN], "gelu") * z[:, HIDDEN:]) @ w2.t() + x
    l = y @ w3.t()
    kept = target >= 0
    loss = torch.where(kept, torch.logsumexp(l, 1) - l.gather(1, target.clamp(min=0)[:, None])[:, 0], torch.zeros_like(l[:, 0]))
    (loss.sum() / target.numel()).backward()
    return loss.detach(), [x.grad] + [v.grad for v in leaves]


def _off(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_gradients(ec):
    """The chain rounds to bf16 seven times on the way to the first weight (h, z, a, y, dy, da, dz and the result), each
    within 2^-8 of a value and mostly less: all together within 8 half steps of the whole, by the norm."""
    model = Model(ec)
    x, t = _data()
    loss, dx, grads = model.gradients(ec, x, t)
    want, exact = _exact(model, x, t)
    assert _off(loss, want) < 8 * 2.0 ** -8
    for name, a, b in zip(("x", "w1", "w2", "w3", "gain", "shift", "b1"), [dx] + grads, exact):
        assert _off(a, b) < 8 * 2.0 ** -8, name


def test_step(ec):
    """The update itself, from the gradients that it was given."""
    model = Model(ec)
    x, t = _data()
    _, _, grads = model.gradients(ec, x, t)
    before = [p.double() for p in model.masters]
    model.step(ec, x, t)
    for p, old, g, decay, w in zip(model.masters, before, grads, [0.1, 0.1, 0.1, 0, 0, 0], model.weights + [None] * 3):
        zero = torch.zeros_like(old)
        want, tol = tr.adamw(old, g.double(), zero, zero, 1, 0.01, (0.9, 0.999), 1e-8, decay)["p"]
        assert bool(((p.double() - want).abs() <= tol).all())
        assert w is None or torch.equal(w, p.bfloat16())


@pytest.mark.parametrize("state", [torch.float32, torch.uint8], ids=str)
def test_captured_step(ec, state):
    """Whole steps replayed from a graph, and the same steps run one by one."""
    one, two = Model(ec, state), Model(ec, state)
    x, t = _data()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one.step(ec, x, t)
    side.synchronize()
    two.step(ec, x, t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = one.step(ec, x, t)
    for k in range(3):
        nx, nt = _data(10 + k)
        x.copy_(nx)
        t.copy_(nt)
        graph.replay()
        torch.cuda.synchronize()
        want = two.step(ec, x, t)
        torch.cuda.synchronize()
        assert torch.equal(got, want), "replay %d" % k
        assert all(torch.equal(a, b) for a, b in zip(one.masters + one.weights, two.masters + two.weights)), "replay %d" % k


def test_two_at_once(ec):
    """Two models step on two streams at the same time: as one after the other."""
    models = [Model(ec, torch.uint8, seed) for seed in (1, 2)]
    alone = [Model(ec, torch.uint8, seed) for seed in (1, 2)]
    data = [_data(3), _data(4)]
    streams = [torch.cuda.Stream() for _ in models]
    torch.cuda.synchronize()
    for k in range(4):
        for model, (x, t), s in zip(models, data, streams):
            with torch.cuda.stream(s):
                model.step(ec, x, t)
    torch.cuda.synchronize()
    for model, (x, t) in zip(alone, data):
        for k in range(4):
            model.step(ec, x, t)
    for a, b in zip(models, alone):
        assert all(torch.equal(p, q) for p, q in zip(a.masters + a.weights, b.masters + b.weights))
        assert torch.equal(a.state.m, b.state.m) and torch.equal(a.state.v, b.state.v)


def test_states_travel_coded(ec):
    """An optimizer's e4m3 states are tensor bytes like any other: coded and decoded they are the same."""
    model = Model(ec, torch.uint8)
    x, t = _data()
    for k in range(3):
        model.step(ec, x, t)
    for s in (model.state.m, model.state.v):
        counts = ec.byte_histogram(s)[0].cpu().tolist()
        cb = ec.Codebook.huffman(counts)
        out, out_len, status = ec.encode(cb, s, 4096)
        back, status2 = ec.decode(cb, out[: int(out_len.item())], s.numel())
        torch.cuda.synchronize()
        assert int(status) == int(status2) == 0 and torch.equal(back, s) and int(out_len) < s.numel()


@pytest.mark.parametrize("m,n,k", [(2048, 1600, 4096), (4100, 1537, 2049), (1600, 8200, 2048), (6000, 2048, 264)])
def test_long_contractions(ec, m, n, k):
    """The backward products of long contractions, which run in tiles of their own, split and not."""
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    dy, w, x = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((m, n), (n, k), (m, k)))
    dx, dw, _ = ec.linear_backward(dy, x, w, need_db=False, dw_dtype=torch.float32)
    _ffn.near(dx, *_ffn.grad_input(dy, w), "dx")
    _ffn.near(dw, *_ffn.grad_weight(dy, x, torch.float32), "dw")
    again = ec.linear_backward(dy, x, w, need_db=False, dw_dtype=torch.float32)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


def test_far_rows(ec):
    """Rows of the contraction 32.4 MiB apart: 32 of them are within 2 GiB, 64 are not."""
    m, n, k, stride = 8192, 1600, 2048, 17_000_000
    g = torch.Generator(device="cuda").manual_seed(5)
    w = torch.empty((n - 1) * stride + k, dtype=torch.bfloat16, device="cuda").as_strided((n, k), (stride, 1))
    w.copy_(torch.randn((n, k), generator=g, device="cuda"))
    dy = torch.randn((m, n), generator=g, device="cuda").bfloat16()
    dx = ec.linear_backward(dy, None, w, need_dw=False, need_db=False)[0]
    assert torch.equal(dx, ec.linear_backward(dy, None, w.contiguous(), need_dw=False, need_db=False)[0])
    _ffn.near(dx[::97], *_ffn.grad_input(dy[::97], w), "dx")


def test_example(ec):
    """examples/feed_forward.py's gated model runs, and its gradients are those of the formulas."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(root, "examples", "feed_forward.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    model = example.GatedModel(WIDTH, HIDDEN, VOCABULARY)
    x, t = _data()
    loss, grads = model.gradients(x, t)
    leaves = [v.double().requires_grad_() for v in model.weights + model.masters[3:]]
    w1, w2, vocabulary, gain, shift = leaves
    h = torch.nn.functional.layer_norm(x.double(), (WIDTH,), gain, shift)
    z = h @ w1.t()
    y = (tr.act(z[:, :HIDDEN], "gelu") * z[:, HIDDEN:]) @ w2.t() + x.double()
    want = torch.nn.functional.cross_entropy(y @ vocabulary.t(), t)
    want.backward()
    assert abs(float(loss) / float(want.detach()) - 1) < 8 * 2.0 ** -8
    for a, b in zip(grads, leaves):
        assert _off(a, b.grad) < 8 * 2.0 ** -8          # as in test_gradients
    before = [p.clone() for p in model.masters]
    model.step(x, t)
    assert not any(torch.equal(p, q) for p, q in zip(before, model.masters))
    assert all(torch.equal(w, p.bfloat16()) for w, p in zip(model.weights, model.masters))
    plain, coded = model.coded_state()
    assert plain == 2 * model.state.m.numel() and 0 < coded
