"""Muon: momentum, orthogonalised update and weights against 64 bits."""
import pytest
import torch

import sparse_ctr_embedding_gb300 as E
from muon_ref import momentum, orthogonal

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    E.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def updates(shapes, grads, m, products="half", beta=0.95, nesterov=True):
    """The orthogonalised updates themselves: a step of rate and scale 1 from weights of 0 leaves their negatives."""
    p = [torch.zeros(s, device="cuda") for s in shapes]
    opt = E.Muon(p, lr=1.0, momentum=beta, nesterov=nesterov, scale=[1.0] * len(p), products=products)
    opt.load_state(m)
    opt.step(grads)
    assert E.emb_check_op_flag() == 0
    return [-x.double() for x in p], opt


def data(shapes, seed=0, rank=None, t=F32):
    g = torch.Generator().manual_seed(seed)
    grads, ms = [], []
    for r, c in shapes:
        x = torch.randn(r, c, generator=g) if rank is None else torch.randn(r, rank, generator=g) @ torch.randn(rank, c, generator=g)
        grads.append((x * 1e-3).to(t).cuda())
        ms.append((torch.randn(r, c, generator=g) * 3e-4).cuda())
    return grads, ms


SHAPES = [[(1, 1)], [(1, 300)], [(300, 1)], [(7, 5)], [(64, 64)], [(128, 128)], [(128, 256)], [(129, 127)], [(200, 1000)], [(1000, 200)],
          [(257, 640)], [(513, 513)], [(1001, 333)], [(384, 2049)], [(2049, 384)], [(1024, 1024)],
          [(33, 70), (256, 512), (1, 9), (130, 64), (640, 640), (512, 1024)]]


@pytest.mark.parametrize("products,planes", [("half", 1), ("split", 2)])
@pytest.mark.parametrize("shapes", SHAPES, ids=str)
def test_update(shapes, products, planes):
    grads, m = data(shapes, seed=len(shapes) + shapes[0][0])
    got, opt = updates(shapes, grads, m, products)
    for o, g, m0, m1, s in zip(got, grads, m, opt.m, shapes):
        want_m, u = momentum(g, m0, 0.95)
        assert float((m1.double() - want_m).abs().max()) <= 3 * 2.0 ** -24 * float(want_m.abs().max() + g.abs().max())
        exact, rounded = orthogonal(u), orthogonal(u, planes)
        far = float((rounded - exact).norm()) + 64 * 2.0 ** -24 * float(exact.norm())
        assert float((o - exact).norm()) <= 3 * far, s
        if min(s) > 1:
            sv = torch.linalg.svdvals(o)
            assert float(sv.max()) < 1.3


def test_larger_updates():
    shapes = [(1024, 4096), (1536, 1100)]
    grads, m = data(shapes, seed=5, t=BF16)
    for products, planes in (("half", 1), ("split", 2)):
        got, _ = updates(shapes, grads, m, products)
        for o, g, m0, s in zip(got, grads, m, shapes):
            u = momentum(g, m0, 0.95)[1]
            exact, rounded = orthogonal(u), orthogonal(u, planes)
            far = float((rounded - exact).norm()) + 64 * 2.0 ** -24 * float(exact.norm())
            assert float((o - exact).norm()) <= 3 * far, (s, products)


@pytest.mark.parametrize("products,planes", [("half", 1), ("split", 2)])
def test_low_rank(products, planes):
    """Directions that the update has only from rounding noise are raised by the steps, in the rounded form alike.
    float32 adds to it: up to four roundings a step of values with |X| = 1 (u each, u = 2^-24), which the steps that
    follow magnify by up to 3.4445 each: 485 from the first one, 683 with the others' (a geometric series)."""
    shapes = [(256, 384), (384, 256)]
    grads, _ = data(shapes, seed=2, rank=6)
    m = [torch.zeros(s, device="cuda") for s in shapes]
    got, _ = updates(shapes, grads, m, products, beta=0.0)
    for o, g in zip(got, grads):
        exact, rounded = orthogonal(g.double()), orthogonal(g.double(), planes)
        assert float((o - exact).norm()) <= 3 * float((rounded - exact).norm()) + 4 * 683 * 2.0 ** -24


@pytest.mark.parametrize("param,grad", [(F32, F32), (BF16, BF16), (F16, F32), (F32, F16), (BF16, F32)])
@pytest.mark.parametrize("nesterov", [True, False])
def test_step(param, grad, nesterov):
    shapes = [(96, 200), (200, 96), (65, 65)]
    grads, m = data(shapes, seed=3, t=grad)
    g = torch.Generator().manual_seed(9)
    p = [(torch.randn(s, generator=g) * 0.05).to(param).cuda() for s in shapes]
    want = [x.double() for x in p]
    ms = [x.double() for x in m]
    scale = torch.tensor(0.5, device="cuda")
    opt = E.Muon(p, lr=0.02, momentum=0.9, weight_decay=0.1, nesterov=nesterov, products="split")
    opt.load_state(m)
    for _ in range(2):
        before = [x.double() for x in p]
        opt.step(grads, grad_scale=scale)
        for i, s in enumerate(shapes):
            ms[i], u = momentum(grads[i].double() * 0.5, ms[i], 0.9, nesterov)
            want[i] = before[i] * (1 - 0.02 * 0.1) - 0.02 * 0.2 * max(s) ** 0.5 * orthogonal(u)
            ulp = torch.finfo(param).eps / 2
            tol = ulp * want[i].abs() + 1e-4 * 0.02 * 0.2 * max(s) ** 0.5 * orthogonal(u).abs().max() + 4 * 2.0 ** -24 * before[i].abs() + 2.0 ** -25
            assert bool(((p[i].double() - want[i]).abs() <= tol).all()), (i, float((p[i].double() - want[i]).abs().max()))


def test_repeats_bitwise_and_many_matrices():
    """More matrices than one launch takes, some of them empty."""
    g = torch.Generator().manual_seed(4)
    shapes = [(int(torch.randint(1, 90, (1,), generator=g)), int(torch.randint(1, 90, (1,), generator=g))) for _ in range(150)]
    shapes[7], shapes[140] = (0, 5), (5, 0)
    shapes.append((700, 900))
    grads, m = data(shapes, seed=6)
    one, _ = updates(shapes, grads, m)
    two, _ = updates(shapes, grads, m)
    for a, b, gr, m0, s in zip(one, two, grads, m, shapes):
        assert torch.equal(a, b)
        if 0 not in s:
            u = momentum(gr, m0, 0.95)[1]
            exact, rounded = orthogonal(u), orthogonal(u, 1)
            assert float((a - exact).norm()) <= 3 * float((rounded - exact).norm()) + 1e-4 * float(exact.norm()), s


def test_zero_and_non_finite_gradients():
    shapes = [(40, 60), (40, 60), (40, 60), (200, 150), (40, 60)]
    grads, _ = data(shapes, seed=7)
    grads[0].zero_()
    grads[1][3, 4] = float("nan")
    grads[2][39, 59] = float("inf")
    grads[4].fill_(3e38)                  # the squares' sum is past float32
    m = [torch.zeros(s, device="cuda") for s in shapes]
    got, _ = updates(shapes, grads, m, beta=0.0)
    assert bool((got[0] == 0).all())
    assert bool(torch.isnan(got[1]).all()) and bool(torch.isnan(got[2]).all()) and bool(torch.isnan(got[4]).all())
    assert bool(torch.isfinite(got[3]).all()) and float(got[3].abs().max()) > 0.01


def test_graph_stream_and_moved_parameters():
    shapes = [(256, 512), (130, 70)]
    grads, m = data(shapes, seed=8, t=BF16)
    make = lambda: [torch.full(s, 0.5, device="cuda") for s in shapes]  # noqa: E731
    p, q, r = make(), make(), make()
    opts = [E.Muon(x, lr=0.01, weight_decay=0.1) for x in (p, q, r)]
    for o in opts:
        o.load_state(m)
    for _ in range(3):
        opts[0].step(grads)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    opts[1].step(grads, stream=s)
    s.synchronize()
    opts[1].params[0].data = opts[1].params[0].data.clone()
    opts[1].m[1] = opts[1].m[1].clone()
    for _ in range(2):
        opts[1].step(grads)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opts[2].step(grads)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(p, opts[1].params, r):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("products", ["half", "split"])
def test_a_wait_that_runs_out(products):
    """The weights stay as they were, the flag is raised once, and the next step is right."""
    shapes = [(300, 700), (1000, 640)]
    grads, m = data(shapes, seed=9)
    want, _ = updates(shapes, grads, m, products)
    for role in ("load", "product", "other"):
        for step in (0, 1, 2):
            p = [torch.full(s, 0.25, device="cuda") for s in shapes]
            opt = E.Muon(p, lr=1.0, scale=[1.0, 1.0], products=products)
            opt.load_state(m)
            try:
                E.emb_debug_lose_op_wait(role, step)
                opt.step(grads)
            finally:
                E.emb_debug_lose_op_wait(None)
            assert E.emb_check_op_flag() == E.EMB_FLAG_OP_TIMEOUT, (role, step)
            assert E.emb_check_op_flag() == 0
            assert all(bool((x == 0.25).all()) for x in p)
            got, _ = updates(shapes, grads, m, products)
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_overlapping_matrices_are_refused():
    p = torch.zeros(8, 16, device="cuda")
    for other in (p, p[2:4], p[7:]):
        with pytest.raises(ValueError, match="overlap"):
            E.Muon([p, other])
    E.Muon([p[:4], p[4:], torch.zeros(0, 5, device="cuda")])      # side by side


@pytest.mark.parametrize("beta", [0.95, 0.99, 0.999])
def test_momentum_near_one(beta):
    """Each of m = beta m + (1 - beta) g's two terms has two roundings, the coefficient's and the product's, and the sum one:
    3 u of the terms' magnitudes, u = 2^-24, and a u for what is of second order.  The update's direction then follows
    within what its own products cost, also where the gradient is only as large as the momentum in it."""
    shapes = [(96, 200), (200, 96), (33, 65)]
    grads, m = data(shapes, seed=11)
    m = [x * (1 - beta) for x in m]                # the new gradient counts for as much as what was there
    m[1].zero_()
    got, opt = updates(shapes, grads, m, "split", beta=beta)
    for o, g, m0, m1 in zip(got, grads, m, opt.m):
        want, u = momentum(g, m0, beta)
        size = beta * m0.double().abs() + (1 - beta) * g.double().abs()
        assert bool(((m1.double() - want).abs() <= 4 * 2.0 ** -24 * size).all()), float(((m1.double() - want).abs() / size).max() * 2 ** 24)
        exact, rounded = orthogonal(u), orthogonal(u, 2)
        far = float((rounded - exact).norm()) + 64 * 2.0 ** -24 * float(exact.norm())
        assert float((o - exact).norm()) <= 3 * far


def test_changes_over_the_same_memory():
    """Other strides, types, scales or products at an address that stays: a step follows them or refuses, with
    nothing changed."""
    shapes = [(64, 64), (48, 80)]
    grads, m = data(shapes, seed=12)

    def step(p, products="half", scale=(1.0, 1.0), m=m):
        opt = E.Muon(p, lr=0.5, scale=scale, products=products)
        opt.load_state(m)
        return opt
    p = [torch.full(s, 0.25, device="cuda") for s in shapes]
    opt = step(p)
    opt.step(grads)
    kept, moved = [x.clone() for x in p], [x.clone() for x in opt.m]
    for change, back in ((lambda: setattr(p[0], "data", p[0].data.t()), lambda: setattr(p[0], "data", p[0].data.t())),
                         (lambda: opt.m.__setitem__(0, opt.m[0].t()), lambda: opt.m.__setitem__(0, opt.m[0].t())),
                         (lambda: opt.m.__setitem__(1, opt.m[1].view(torch.int32)), lambda: opt.m.__setitem__(1, opt.m[1].view(F32))),
                         (lambda: setattr(p[1], "data", p[1].data.view(80, 48)), lambda: setattr(p[1], "data", p[1].data.view(48, 80))),
                         (lambda: setattr(opt, "scale", [1.0]), lambda: setattr(opt, "scale", [1.0, 1.0]))):
        change()
        with pytest.raises((ValueError, TypeError)):
            opt.step(grads)
        back()
        assert all(map(torch.equal, p, kept)) and all(map(torch.equal, opt.m, moved))
    opt.step(grads)                                            # as it was
    want = [torch.full(s, 0.25, device="cuda") for s in shapes]
    ref = step(want)
    ref.step(grads)
    ref.step(grads)
    assert all(map(torch.equal, p, want)) and all(map(torch.equal, opt.m, ref.m))
    # the same bytes as another type of its size
    a, b = [[torch.full(s, 0.25, dtype=BF16, device="cuda") for s in shapes] for _ in range(2)]
    oa, bits = step(a), a[0].data
    oa.step(grads)
    a[0].data = bits.view(F16)
    ob = step(b)
    ob.step(grads)
    ob = step([b[0].data.view(F16), b[1]], m=ob.m)
    oa.step(grads)
    ob.step(grads)
    assert a[0].dtype == F16 and torch.equal(a[0], ob.params[0]) and torch.equal(a[1], b[1])
    # scale and products
    a, b, c = [[torch.full(s, 0.25, device="cuda") for s in shapes] for _ in range(3)]
    oa, ob, oc = step(a), step(b, "split", (2.0, 0.5)), step(c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        oa.step(grads)
    old = oa.workspace.data_ptr()
    oa.products, oa.scale = "split", [2.0, 0.5]
    oa.step(grads)
    ob.step(grads)
    assert oa.workspace.data_ptr() != old and all(map(torch.equal, a, b)) and all(map(torch.equal, oa.m, ob.m))
    for x, y in zip(a + oa.m, c + oc.m):
        x.copy_(y)
    other = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")      # would lie where the graph's workspace was
    graph.replay()
    oc.step(grads)
    torch.cuda.synchronize()
    assert all(map(torch.equal, a, c)) and all(map(torch.equal, oa.m, oc.m)) and bool((other == 255).all())
    assert E.emb_check_op_flag() == 0


@pytest.mark.parametrize("products", ["half", "split"])
def test_momenta_after_a_wait_that_ran_out(products):
    """The momenta have taken the gradients, the weights have not: repeated after the momenta were set back the step
    is the one that was lost; repeated as things are, it counts the gradients twice."""
    shapes = [(300, 700), (64, 100)]
    grads, m = data(shapes, seed=13)
    make = lambda: E.Muon([torch.full(s, 0.25, device="cuda") for s in shapes], lr=0.1, products=products)  # noqa: E731
    ref = make()
    ref.load_state(m)
    ref.step(grads)
    once = [x.clone() for x in ref.m]
    twice = make()
    twice.load_state(once)
    twice.step(grads)
    for role in ("load", "product", "other"):
        opts = [make(), make()]
        for opt in opts:
            opt.load_state(m)
            try:
                E.emb_debug_lose_op_wait(role, 1)
                opt.step(grads)
            finally:
                E.emb_debug_lose_op_wait(None)
            assert E.emb_check_op_flag() == E.EMB_FLAG_OP_TIMEOUT
            assert all(bool((x == 0.25).all()) for x in opt.params) and all(map(torch.equal, opt.m, once))
        opts[0].load_state(m)
        for opt, want in zip(opts, (ref, twice)):
            opt.step(grads)
            assert all(map(torch.equal, opt.m, want.m)) and all(map(torch.equal, opt.params, want.params))
        assert E.emb_check_op_flag() == 0
