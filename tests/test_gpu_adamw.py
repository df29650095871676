"""AdamW over many tensors against its 64-bit form: states in fp32 and e4m3."""

import pytest

torch = pytest.importorskip("torch")

import _training as tr  # noqa: E402
from _ffn import near, values  # noqa: E402

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
BLOCK = 256


@pytest.fixture(scope="module")
def ec():
    import lossless_entropy_coding_amd as ec
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ec.lib()
    return ec


def _tensors(shapes, seed=0, grad=torch.bfloat16, size=1e-2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ps = [torch.randn(s, generator=g, device="cuda") * 0.1 for s in shapes]
    gs = [(torch.randn(s, generator=g, device="cuda") * size * torch.exp(torch.randn(s, generator=g, device="cuda"))).to(grad)
          for s in shapes]
    return ps, gs


def _blocks(n):
    return -(-n // BLOCK)


def _places(shapes):
    at, found = 0, []
    for s in shapes:
        n = 1
        for v in s:
            n *= v
        found.append((at, n))
        at += _blocks(n) * BLOCK
    return found, at


SHAPES = [
    [(1,)], [(256,)], [(257,)], [(255,), (1,), (4096,)], [(3, 5, 7), (0,), (64, 129)], [(4096 * 3 + 17,)],
    [(300 + 37 * i,) for i in range(130)],
]


@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("copies", [False, True])
@pytest.mark.parametrize("shapes", SHAPES, ids=lambda s: "%d tensors from %s" % (len(s), s[0]))
def test_fp32(ec, shapes, copies, grad):
    ps, _ = _tensors(shapes)
    state = ec.adamw_state(ps)
    cs = [torch.zeros_like(p, dtype=torch.bfloat16) for p in ps] if copies else None
    places, total = _places(shapes)
    assert state.m.numel() == total
    m = v = None
    lr, betas, eps = 0.01, (0.9, 0.99), 1e-6
    scale = torch.full((1,), 0.5, device="cuda")
    decays = [0.1 * (i % 3) for i in range(len(ps))]
    for step in range(1, 4):
        gs = _tensors(shapes, seed=step, grad=grad)[1]
        before = [(p.double(), *(t[a:a + n].double().view(p.shape) for t in (state.m, state.v))) for p, (a, n) in zip(ps, places)]
        ec.adamw(ps, gs, state, lr=lr, betas=betas, eps=eps, weight_decay=decays, grad_scale=scale, copies=cs)
        assert int(state.steps) == step
        for i, (p, g, (a, n)) in enumerate(zip(ps, gs, places)):
            want = tr.adamw(before[i][0], g.double(), before[i][1], before[i][2], step, lr, betas, eps, decays[i], 0.5)
            near(p, *want["p"], "p of %d, step %d" % (i, step))
            near(state.m[a:a + n].view(p.shape), *want["m"], "m")
            near(state.v[a:a + n].view(p.shape), *want["v"], "v")
            for t in (state.m, state.v):
                assert bool((t[a + n:a + _blocks(n) * BLOCK] == 0).all())
            if copies:
                assert torch.equal(cs[i], p.bfloat16())
    assert m is v is None


@pytest.mark.parametrize("kind", [F8, torch.uint8], ids=str)
@pytest.mark.parametrize("shapes", SHAPES, ids=lambda s: "%d tensors from %s" % (len(s), s[0]))
def test_e4m3(ec, shapes, kind):
    """p as from the states' values; each state on the value that its random bits choose (unless the choice is within
    2^-13 of the other one, more than a 32-bit value with its errors moves it: 16 steps of a value, 8 u each)."""
    ps, _ = _tensors(shapes)
    state = ec.adamw_state(ps, kind)
    places, total = _places(shapes)
    lr, betas, eps, seed = 0.01, (0.9, 0.99), 1e-6, 12345
    for step in range(1, 6):
        gs = _tensors(shapes, seed=step)[1]
        old_m, old_v = tr.held(state, "m"), tr.held(state, "v")
        before = [p.double() for p in ps]
        ec.adamw(ps, gs, state, lr=lr, betas=betas, eps=eps, weight_decay=0.1, seed=seed)
        um, uv = (u.cuda() for u in tr.random_shares(seed, step, 0, total))
        new_m, new_v = torch.zeros(total, device="cuda", dtype=torch.float64), torch.zeros(total, device="cuda", dtype=torch.float64)
        for i, (p, g, (a, n)) in enumerate(zip(ps, gs, places)):
            s = slice(a, a + n)
            want = tr.adamw(before[i].view(-1), g.double().view(-1), old_m[s], old_v[s], step, lr, betas, eps, 0.1)
            near(p.view(-1), *want["p"], "p of %d, step %d" % (i, step))
            new_m[s], new_v[s] = want["m"][0], want["v"][0]
        for name, new, u in (("m", new_m, um), ("v", new_v, uv)):
            if not total:
                continue
            want, scale, margin, near_grid = tr.random_rounding(new, u, name == "v")
            got, got_scale = values(getattr(state, name)), getattr(state, name + "_scale").double()
            sure = (margin > 2.0 ** -13) & (near_grid > 2.0 ** -13) | (new == 0)
            # a block's scale too may fall either way where its largest value is next to a border
            top = (new.abs().sqrt() if name == "v" else new.abs()).view(-1, BLOCK).amax(1)
            firm = ((top / scale / 448 - 1).abs() > 1e-5) & ((top / scale / 224 - 1).abs() > 1e-5)
            assert torch.equal(got_scale[firm], scale[firm])
            assert firm.numel() < 100 or float(firm.double().mean()) > 0.9      # one block may well lie there
            # 0.9 of ten steps of the grid is nine: where the gradient is small a moved value lies on the grid again
            assert total < 5000 or float(sure.double().mean()) > 0.8
            sure &= firm.repeat_interleave(BLOCK)
            assert torch.equal(got[sure], want[sure]), "%s, step %d" % (name, step)
        for (a, n) in places:
            for t in (state.m, state.v):
                assert bool((t.view(torch.uint8)[a + n:a + _blocks(n) * BLOCK] == 0).all())


def test_means_are_kept(ec):
    """Over many seeds the mean of a held value is the value: m's and v's roundings are as often up as their place says.
    The mean of 400 draws of a variable that lies within one step (of v: between two squares of the grid) is off by more
    than 5 / sqrt(400) of half a step in less than one of 10^6; of 1024 values none is expected."""
    n, draws = 1024, 400
    ps, gs = _tensors([(n,)], seed=3)
    start = ec.adamw_state(ps, F8)
    ec.adamw([p.clone() for p in ps], gs, start, seed=1)
    base = [t.clone() for t in start]
    sums = {"m": torch.zeros(n, device="cuda", dtype=torch.float64), "v": torch.zeros(n, device="cuda", dtype=torch.float64)}
    top = {}
    for seed in range(draws):
        state = ec.AdamWState(*(t.clone() for t in base))
        ec.adamw([p.clone() for p in ps], gs, state, seed=1000 + seed)
        for name in sums:
            x = tr.held(state, name)
            sums[name] += x / draws
            lo, hi = top.get(name, (x, x))
            top[name] = (torch.minimum(lo, x), torch.maximum(hi, x))
    old = ec.AdamWState(*base)
    want = tr.adamw(ps[0].double(), gs[0].double(), tr.held(old, "m"), tr.held(old, "v"), 2, 1e-3, (0.9, 0.999), 1e-8, 0.01)
    for name in sums:
        lo, hi = top[name]
        value = want[name][0]
        room = 5 / draws ** 0.5 * 0.5 * (hi - lo) + 1e-5 * value.abs()
        # where every draw gave the same value the other one is rarer than one in 20
        room = torch.where(hi > lo, room, 0.3 * value.abs() * 20 / draws + 2.0 ** -10 * getattr(old, name + "_scale").double().repeat_interleave(BLOCK))
        assert bool(((sums[name] - value).abs() <= room).all()), name


def test_steady_gradient(ec):
    """With one gradient, m and v go to it and to its square although a step moves them by less than e4m3 can hold
    (beta2 0.999: a thousandth), so that the change of p stays lr: held to the nearest value, v would stop after some ten
    steps.  After 600 steps the mean of v over 4096 values is g^2 (1 - 0.999^600) within 5 %: a value's own spread is
    near a third, and 5 deviations of the mean of 4096 are 2.6 %."""
    n = 4096
    p = torch.zeros(n, device="cuda")
    g = torch.full((n,), 0.01, device="cuda")
    state = ec.adamw_state([p], F8)
    for k in range(600):
        ec.adamw([p], [g], state, weight_decay=0.0, seed=7)
    want = 1e-4 * (1 - 0.999 ** 600)
    assert abs(float(tr.held(state, "v").mean()) / want - 1) < 0.05
    assert abs(float(tr.held(state, "m").mean()) / 0.01 - 1) < 0.02


def test_fixed_by_seed_step_and_place(ec):
    ps, gs = _tensors([(5000,), (77,)], seed=5)

    def run(seed, steps=0):
        qs = [p.clone() for p in ps]
        state = ec.adamw_state(qs, F8)
        state.steps.fill_(steps)
        ec.adamw(qs, gs, state, seed=seed)
        return [t.view(torch.uint8).clone() for t in (state.m, state.v)] + qs

    a, b, c = run(1), run(1), run(2)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert not torch.equal(a[0], c[0]) and not torch.equal(a[1], c[1])
    assert torch.equal(a[2], c[2])              # p goes by the values before they are rounded
    assert not torch.equal(a[0], run(1, steps=3)[0])


@pytest.mark.parametrize("kind", [torch.float32, F8], ids=str)
def test_special_values(ec, kind):
    """What is not finite stays where it is; the rest of its block is as without it."""
    ps, gs = _tensors([(600,)], seed=6, grad=torch.float32)
    want, clean = [p.clone() for p in ps], ec.adamw_state(ps, kind)
    gs0 = [g.clone() for g in gs]
    for i in (3, 4, 300):
        gs0[0][i] = 0.0
    ec.adamw(want, gs0, clean)
    gs[0][3], gs[0][4], gs[0][300] = float("nan"), float("inf"), float("-inf")
    got, state = [p.clone() for p in ps], ec.adamw_state(ps, kind)
    ec.adamw(got, gs, state)
    rest = torch.ones(600, dtype=torch.bool, device="cuda")
    rest[[3, 4, 300]] = False
    assert torch.equal(got[0][rest], want[0][rest]) and not bool(got[0][~rest].isfinite().any())
    for name in ("m", "v"):
        a, b = values(getattr(state, name))[:600], values(getattr(clean, name))[:600]
        assert torch.equal(a[rest], b[rest]) and not bool(a[~rest].isfinite().any())
    if kind == F8:
        assert torch.equal(state.m_scale, clean.m_scale) and torch.equal(state.v_scale, clean.v_scale)


@pytest.mark.parametrize("kind", [torch.float32, F8], ids=str)
def test_extremes(ec, kind):
    """Gradients of zero, tiny and huge ones (their squares within fp32)."""
    n = 256
    for size in (0.0, 1e-30, 1e-20, 1e15):
        p = torch.ones(n, device="cuda")
        g = torch.full((n,), size, device="cuda")
        g[::2] *= -1
        state = ec.adamw_state([p], kind)
        ec.adamw([p], [g], state, lr=0.1, weight_decay=0.0)
        want = tr.adamw(torch.ones(n, device="cuda").double(), g.double(), 0 * g.double(), 0 * g.double(), 1, 0.1, (0.9, 0.999), 1e-8,
                        0.0)
        # squares below fp32's normal range keep fewer digits; eps is far above their roots
        near(p, want["p"][0], want["p"][1] + 1e-9, "size %g" % size)
        if kind == torch.float32:
            near(state.m[:n], want["m"][0], want["m"][1] + 1e-44)
            near(state.v[:n], want["v"][0], want["v"][1] + 3e-45)
        else:
            assert bool(values(state.m).isfinite().all()) and bool(values(state.v).isfinite().all())
            m = tr.held(state, "m")[:n]
            assert bool(((m - want["m"][0]).abs() <= want["m"][0].abs() / 8 + 2.0 ** -69).all())


def test_views_at_odd_places(ec):
    """Params, gradients and copies that begin anywhere in a larger buffer; what lies between them stays."""
    n = [1000, 513, 7]
    flat, flat_g, flat_c = (torch.full((2000,), 9.0, device="cuda", dtype=t) for t in (torch.float32, torch.bfloat16, torch.bfloat16))
    at, ps, gs, cs, qs = 1, [], [], [], []
    ref, ref_g = _tensors([(v,) for v in n], seed=8)
    kept = torch.ones(2000, dtype=torch.bool, device="cuda")
    for r, rg, v in zip(ref, ref_g, n):
        s = slice(at, at + v)
        flat[s], flat_g[s] = r, rg
        ps.append(flat[s])
        gs.append(flat_g[s])
        cs.append(flat_c[s])
        qs.append(r.clone())
        kept[s] = False
        at += v + 3
    for kind in (torch.float32, F8):
        one, two = ec.adamw_state(ps, kind), ec.adamw_state(qs, kind)
        copies = [None, cs[1], None]
        ec.adamw(ps, gs, one, copies=copies)
        ec.adamw(qs, ref_g, two)
        for p, q in zip(ps, qs):
            assert torch.equal(p, q)
        for a, b in zip(one[:2], two[:2]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(cs[1], qs[1].bfloat16()) and bool((cs[0] == 9).all()) and bool((cs[2] == 9).all())
        assert bool((flat[kept] == 9).all()) and bool((flat_g[kept] == 9).all())


def test_mixed_gradients(ec):
    ps, gs = _tensors([(400,), (900,), (64, 5)], seed=9)
    gs[1] = gs[1].float()
    a, b = [p.clone() for p in ps], [p.clone() for p in ps]
    one, two = ec.adamw_state(a), ec.adamw_state(b)
    ec.adamw(a, gs, one)
    ec.adamw(b, [g.float() for g in gs], two)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(one.m, two.m) and torch.equal(one.v, two.v)


def test_learning_rate_tensor_and_late_steps(ec):
    for steps in (0, 1, 10, 1000, 10 ** 6, 2 ** 30):
        ps, gs = _tensors([(500,)], seed=10)
        a, b = [p.clone() for p in ps], [p.clone() for p in ps]
        one, two = ec.adamw_state(a), ec.adamw_state(b)
        for s in (one, two):
            s.steps.fill_(steps)
        ec.adamw(a, gs, one, lr=torch.full((1,), 0.003, device="cuda"))
        ec.adamw(b, gs, two, lr=0.003)
        assert torch.equal(a[0], b[0]) and int(one.steps) == steps + 1
        z = torch.zeros(500, device="cuda", dtype=torch.float64)
        near(a[0], *tr.adamw(ps[0].double(), gs[0].double(), z, z, steps + 1, 0.003, (0.9, 0.999), 1e-8, 0.01)["p"], str(steps))


@pytest.mark.parametrize("kind", [torch.float32, F8], ids=str)
def test_stream_and_graph(ec, kind):
    """A captured step goes on from step to step as eager ones do."""
    shapes = [(3000,), (100, 33), (5,)]
    ps, gs = _tensors(shapes, seed=11)
    qs = [p.clone() for p in ps]
    one, two = ec.adamw_state(ps, kind), ec.adamw_state(qs, kind)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ec.adamw(ps, gs, one, stream=side)
    side.synchronize()
    ec.adamw(qs, gs, two)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ec.adamw(ps, gs, one, seed=3)
    for k in range(4):
        for g, new in zip(gs, _tensors(shapes, seed=20 + k)[1]):
            g.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        ec.adamw(qs, gs, two, seed=3)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(ps, qs)), "replay %d" % k
        assert int(one.steps) == int(two.steps) == k + 2
        for a, b in zip(one[:2], two[:2]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_more_values_than_a_launch(ec):
    """A tensor whose state passes 2^32 bytes."""
    n = (1 << 30) + 4096 + 3
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    at = torch.tensor([0, 1, 255, 256, (1 << 30) - 1, 1 << 30, n - 1], device="cuda")
    g[at] = 1.0
    state = ec.adamw_state([p])
    ec.adamw([p], [g], state, lr=0.5, weight_decay=0.0)
    torch.cuda.synchronize()
    assert int((p != 0).sum()) == at.numel() and bool((p[at] < -0.49).all())
    assert int((state.m != 0).sum()) == at.numel() and bool((state.v[at] != 0).all())
