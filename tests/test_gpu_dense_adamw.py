"""AdamW over many tensors against the formula: float32 states in 64 bits, 8-bit
states bit for bit (each operation is one float32 rounding, so any IEEE
evaluation agrees)."""
import pytest
import torch

import sparse_ctr_embedding_gb300 as E
from dense_ref import ROUND, U, adamw32, e4m3_values, random_bits, round_state

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HYPER = (1e-2, 0.9, 0.999, 1e-8, 0.05)


@pytest.fixture(scope="module", autouse=True)
def built():
    E.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def tensors(sizes, pt, gt, seed):
    g = torch.Generator().manual_seed(seed)
    p = [torch.randn(n, generator=g).to(pt) for n in sizes]
    grads = [[(torch.randn(n, generator=g) * 10.0 ** float(torch.randint(-4, 2, (1,), generator=g))).to(gt) for n in sizes]
             for _ in range(3)]
    return p, grads


SIZES = [[1], [255, 256, 257, 0, 1], [100_003, 5, 64], [3] * 45 + [2048], [17] * 400 + [5000], [1_000_000]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("pt,gt", [(F32, F32), (F32, BF16), (BF16, BF16), (F16, F16), (BF16, F32)])
def test_float32_states(sizes, pt, gt):
    """Three steps: bit for bit in float32, and each step from the states before it
    against 64 bits (m and v take three roundings each; a weight its product
    with the decay, the update four, and the difference)."""
    p, grads = tensors(sizes, pt, gt, len(sizes))
    dev = [t.cuda() for t in p]
    opt = E.AdamW(dev, lr=HYPER[0], betas=HYPER[1:3], eps=HYPER[3], weight_decay=HYPER[4])
    m, v = [torch.zeros(n) for n in sizes], [torch.zeros(n) for n in sizes]
    lr, b1, b2, eps, wd = HYPER
    for t in range(1, 4):
        opt.step([g.cuda() for g in grads[t - 1]])
        for i, n in enumerate(sizes):
            g, at = grads[t - 1][i].double(), opt._at[i]
            m0, v0, p0 = m[i].double(), v[i].double(), p[i].double()
            w, m[i], v[i], _ = adamw32(p[i], grads[t - 1][i], m[i], v[i], None, (*HYPER, t), False)
            p[i] = w.to(pt)
            got_m, got_v = opt.arena["m"][at:at + n].cpu(), opt.arena["v"][at:at + n].cpu()
            assert torch.equal(dev[i].cpu(), p[i]) and torch.equal(got_m, m[i]) and torch.equal(got_v, v[i]), (t, i)
            m64, v64 = b1 * m0 + (1 - b1) * g, b2 * v0 + (1 - b2) * g * g
            assert bool(((got_m.double() - m64).abs() <= 4 * U * (b1 * m0.abs() + (1 - b1) * g.abs()) + 2e-45).all())
            assert bool(((got_v.double() - v64).abs() <= 6 * U * v64 + 4e-45).all())
            size = lr / (1 - b1 ** t) * (b1 * m0.abs() + (1 - b1) * g.abs()) / (torch.sqrt(v64 / (1 - b2 ** t)) + eps)
            want = p0 * (1 - lr * wd) - lr * (m64 / (1 - b1 ** t)) / (torch.sqrt(v64 / (1 - b2 ** t)) + eps)
            tol = 4 * U * p0.abs() + 16 * U * size + ROUND[pt] * want.abs() + (2.0 ** -25 if pt == F16 else 1e-40)
            assert bool(((dev[i].cpu().double() - want).abs() <= tol).all()), (t, i)


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("pt,gt", [(F32, F32), (F32, BF16), (F16, F16), (BF16, F16)])
def test_8bit_states_bit_for_bit(sizes, pt, gt):
    p, grads = tensors(sizes, pt, gt, len(sizes) + 1)
    dev = [t.cuda() for t in p]
    opt = E.AdamW(dev, lr=HYPER[0], betas=HYPER[1:3], eps=HYPER[3], weight_decay=HYPER[4], state="q8", seed=11)
    deq = [(torch.zeros(n), torch.zeros(n)) for n in sizes]
    for t in range(1, 4):
        opt.step([g.cuda() for g in grads[t - 1]])
        for i, n in enumerate(sizes):
            w, m, _, u = adamw32(p[i], grads[t - 1][i], deq[i][0], None, deq[i][1], (*HYPER, t), True)
            p[i] = w.to(pt)
            assert torch.equal(dev[i].cpu(), p[i]), (t, i)
            at, blk = opt._at[i], -(-n // 256)
            bits = random_bits(at, n, 11, t)
            qm, sm = round_state(m, bits & 0xFFFF)
            qu, su = round_state(u, bits >> 16)
            qu = torch.where((u > 0) & (qu == 0), torch.full_like(qu, 2.0 ** -9), qu)
            got = {k: x[at:at + n].cpu().float() for k, x in opt.arena.items() if not k.endswith("scale")}
            assert torch.equal(got["m"], qm) and torch.equal(got["v"], qu), (t, i)
            assert torch.equal(opt.arena["m_scale"][at // 256:at // 256 + blk].cpu(), sm)
            assert torch.equal(opt.arena["v_scale"][at // 256:at // 256 + blk].cpu(), su)
            full = lambda s: s.repeat_interleave(256)[:n]  # noqa: E731
            deq[i] = (qm * full(sm), qu * full(su))


def test_stochastic_rounding_is_unbiased_and_slow_averages_move():
    """Over many steps' random numbers the mean stored value is the value: within
    5 standard errors, each stored value one of the codes around it.  And a
    root-mean-square that must fall by 1 - sqrt(0.999) a step falls."""
    n, reps = 2048, 400
    m0 = torch.linspace(0.01, 1.0, n)
    total = torch.zeros(n, dtype=torch.float64)
    vals = e4m3_values().double()
    for r in range(reps):
        dev = torch.zeros(n, device="cuda")
        opt = E.AdamW([dev], lr=0.0, betas=(0.0, 0.0), weight_decay=0.0, state="q8", seed=r)
        opt.step([m0.cuda()])
        got = opt.arena["m"].cpu().float().double()
        scale = opt.arena["m_scale"].cpu().double().repeat_interleave(256)
        x = m0.double() / scale
        lo = (torch.searchsorted(vals, x * (1 + 1e-6), right=True) - 1).clamp(0, 126)
        gap = vals[(lo + 1).clamp_max(126)] - vals[lo]
        assert bool(((got - x).abs() <= gap * (1 + 1e-4) + 1e-4).all())
        total += got * scale - m0.double()
    gap = gap * scale
    # one rounding has variance at most gap^2/4; the float32 scale is good to 2 u
    assert bool((total.abs() / reps <= 5 * gap / 2 / reps ** 0.5 + 8 * U).all())
    dev = torch.zeros(512, device="cuda")
    opt = E.AdamW([dev], lr=0.0, state="q8")
    one = torch.full((512,), 1.0)
    one[::256] = 4.0                 # holds the blocks' scales
    opt.step([one.cuda()])
    for _ in range(700):
        g = torch.zeros(512)
        g[::256] = 4.0
        opt.step([g.cuda()])
    u = (opt.arena["v"].cpu().float() * opt.arena["v_scale"].cpu().repeat_interleave(256))[1:256].double().mean()
    start, fall = (1 - 0.999) ** 0.5, 0.999 ** 350
    assert 0.8 * start * fall < float(u) < 1.25 * start * fall


def test_copies_scale_and_non_finite():
    p, grads = tensors([1000, 300], F32, F32, 5)
    dev, half = [t.cuda() for t in p], [torch.empty(1000, dtype=BF16, device="cuda"), None]
    opt = E.AdamW(dev, lr=HYPER[0], weight_decay=0.0, copies=half)
    twin = [t.cuda() for t in p]
    ref = E.AdamW(twin, lr=HYPER[0], weight_decay=0.0)
    opt.step([g.cuda() for g in grads[0]], grad_scale=torch.tensor([0.25], device="cuda"))
    ref.step([(g * 0.25).cuda() for g in grads[0]])
    for a, b in zip(dev, twin):
        assert torch.equal(a, b)
    assert torch.equal(half[0], dev[0].to(BF16))
    bad = grads[1][0].clone()
    bad[3], bad[600] = float("inf"), float("nan")
    for state in ("f32", "q8"):
        dev = [p[0].cuda()]
        opt = E.AdamW(dev, state=state)
        opt.step([bad.cuda()])
        off = ~torch.isfinite(dev[0].cpu())
        assert off.nonzero().flatten().tolist() == [3, 600]
        if state == "q8":
            assert bool(torch.isfinite(opt.arena["m_scale"]).all() & torch.isfinite(opt.arena["v_scale"]).all())
            code = opt.arena["m"].cpu().float()[:1000]
            assert torch.isnan(code).nonzero().flatten().tolist() == [3, 600]


def test_unaligned_parameters_and_checkpoint():
    g = torch.Generator().manual_seed(3)
    buf = torch.zeros(4001, device="cuda")
    init = torch.randn(4000, generator=g)
    buf[1:] = init.cuda()
    grad = torch.zeros(4001, device="cuda")
    grad[1:] = torch.randn(4000, generator=g).cuda()
    twin = init.cuda()
    a = E.AdamW([buf[1:]], state="q8", seed=2)
    b = E.AdamW([twin], state="q8", seed=2)
    a.step([grad[1:]])
    b.step([grad[1:].clone()])
    assert torch.equal(buf[1:], twin) and torch.equal(a.arena["m"].view(torch.uint8), b.arena["m"].view(torch.uint8))
    # a second optimizer that resumes from the first one's states takes the same step
    c_p = twin.clone()
    c = E.AdamW([c_p], state="q8", seed=2)
    c.load_state(b.step_count, *[[b.arena[k][:n]] for k, n in (("m", 4000), ("v", 4000), ("m_scale", 16), ("v_scale", 16))])
    b.step([grad[1:].clone()])
    c.step([grad[1:].clone()])
    assert torch.equal(twin, c_p) and torch.equal(b.arena["v"].view(torch.uint8), c.arena["v"].view(torch.uint8))


def test_refusals():
    p = torch.zeros(8, device="cuda")
    with pytest.raises(ValueError):
        E.AdamW([])
    with pytest.raises(KeyError):
        E.AdamW([p], state="4bit")
    opt = E.AdamW([p])
    for bad in ([], [torch.zeros(7, device="cuda")], [torch.zeros(8)], [torch.zeros(16, device="cuda")[::2]]):
        with pytest.raises(ValueError):
            opt.step(bad)
    with pytest.raises(TypeError):
        opt.step([torch.zeros(8, dtype=torch.float64, device="cuda")])
    opt = E.AdamW([p], betas=(1.0, 0.9))
    with pytest.raises(E.EmbError) as ei:
        opt.step([p.clone()])
    assert ei.value.name == "EMB_ERR_INVALID_ARG"
    assert opt.step_count == 0


@pytest.mark.parametrize("state", ["f32", "q8"])
def test_parameters_copies_and_states_that_move(state):
    """New storage under the same tensors (p.data = ..., half(), set_(), a replaced
    state): a step updates what the tensors are now, and writes nothing where they were."""
    g = torch.Generator().manual_seed(4)
    init = [torch.randn(n, generator=g) for n in (700, 33, 5)]
    grads = [[torch.randn(n, generator=g).cuda() for n in (700, 33, 5)] for _ in range(5)]

    def start():
        p = [t.cuda() for t in init]
        c = [torch.empty(700, dtype=BF16, device="cuda"), None, None]
        return p, c, E.AdamW(p, lr=1e-2, state=state, seed=1, copies=c)

    p, c, opt = start()
    still_p, still_c, still = start()
    same = lambda: all(torch.equal(a, b) for a, b in zip(p, still_p)) and torch.equal(c[0], still_c[0])  # noqa: E731
    opt.step(grads[0])
    still.step(grads[0])
    assert same()
    kept = [p[0].data, p[1].detach(), c[0].data]     # the storage that the tensors leave
    p[0].data = p[0].data.clone()
    p[1].set_(p[1].clone())
    c[0].data = torch.empty_like(c[0].data)
    before = [t.clone() for t in kept]
    opt.step(grads[1])
    still.step(grads[1])
    assert same() and torch.equal(kept[0], before[0]) and torch.equal(kept[2], before[2])
    old = opt.arena["m"]
    opt.arena["m"] = old.clone()
    seen = old.view(torch.uint8).clone()
    opt.step(grads[2])
    still.step(grads[2])
    assert same() and torch.equal(old.view(torch.uint8), seen)
    for key in opt.arena:
        if opt.arena[key] is not None:
            assert torch.equal(opt.arena[key].view(torch.uint8), still.arena[key].view(torch.uint8)), key
    # a parameter of another type, as module.half() leaves it: the step of an optimizer made for it
    wide = p[2].data
    p[2].data = p[2].data.half()
    twin = [p[2].detach().clone()]
    of = E.AdamW(twin, lr=1e-2, state=state, seed=1)
    at = opt._at[2]
    cut = {k: None if v is None else [v[at // 256:at // 256 + 1] if k.endswith("scale") else v[at:at + 5]] for k, v in opt.arena.items()}
    of.load_state(opt.step_count, **cut)
    of._tensors[0].first = at
    before = wide.clone()
    opt.step(grads[3])
    of.step([grads[3][2]])
    assert torch.equal(p[2], twin[0]) and torch.equal(wide, before)


def test_parameters_that_change_size_or_lose_their_storage_are_refused():
    p = [torch.zeros(300, device="cuda"), torch.zeros(20, device="cuda")]
    opt = E.AdamW(p, state="q8")
    grads = [torch.ones(300, device="cuda"), torch.ones(20, device="cuda")]
    whole = p[0].data
    for other in (torch.zeros(200, device="cuda"), torch.zeros(600, device="cuda")[::2], torch.zeros(300),
                  torch.zeros(300, dtype=torch.float64, device="cuda")):
        p[0].data = other
        with pytest.raises((ValueError, TypeError)):
            opt.step(grads)
        assert opt.step_count == 0 and bool((p[1] == 0).all())
    p[0].data = whole
    q = torch.zeros(40, device="cuda")
    p[1].data = q[20:]
    q.untyped_storage().resize_(0)
    with pytest.raises(ValueError):
        opt.step(grads)
    p[1].data = torch.zeros(20, device="cuda")
    arena = opt.arena["v"]
    for bad in (arena[:256], arena.float(), None):
        opt.arena["v"] = bad
        with pytest.raises((ValueError, TypeError)):
            opt.step(grads)
    opt.arena["v"] = arena
    assert opt.step_count == 0 and bool((p[0] == 0).all())
    opt.step(grads)
    assert bool((p[0] < 0).all()) and bool((p[1] < 0).all())


class Elsewhere(torch.Tensor):
    """A tensor that says it is on GPU 1."""

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        if func == torch.Tensor.get_device:
            return 1
        return super().__torch_function__(func, types, args, kwargs or {})


def test_tensors_on_another_device_are_refused(monkeypatch):
    """A gradient, its scale, a copy or a parameter on another GPU, or another GPU current: nothing is launched."""
    away = lambda t: t.as_subclass(Elsewhere)  # noqa: E731
    z = lambda n, **kw: torch.zeros(n, device="cuda", **kw)  # noqa: E731
    opt = E.AdamW([z(300), z(7)])

    def launched(*a):
        raise AssertionError("launched")

    monkeypatch.setattr(E, "emb_adamw_step", launched)
    for bad in ([z(300), away(z(7))], [away(z(300)), away(z(7))]):
        with pytest.raises(ValueError, match="cuda:0"):
            opt.step(bad)
    with pytest.raises(ValueError, match="cuda:0"):
        opt.step([z(300), z(7)], grad_scale=away(z(1)))
    with pytest.raises(ValueError, match="cuda:0"):
        E.AdamW([z(300), away(z(7))])
    with pytest.raises(ValueError, match="cuda:0"):
        E.AdamW([z(300)], copies=[away(z(300, dtype=BF16))])
    monkeypatch.setattr(E, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="cuda:1"):
        opt.step([z(300), z(7)])
    monkeypatch.undo()
    with pytest.raises(ValueError, match="stream"):
        monkeypatch.setattr(torch.cuda.Stream, "device_index", property(lambda self: 1), raising=False)
        opt.step([z(300), z(7)], stream=torch.cuda.Stream())
    monkeypatch.undo()
    assert opt.step_count == 0
    opt.step([z(300), z(7)], stream=torch.cuda.Stream())
    assert opt.step_count == 1


def test_load_state_takes_all_or_nothing():
    """A refused state leaves the optimizer as it was; lists of another length are refused."""
    for state, keys in (("f32", ("m", "v")), ("q8", ("m", "v", "m_scale", "v_scale"))):
        opt = E.AdamW([torch.zeros(300, device="cuda"), torch.zeros(5, device="cuda")], state=state)
        opt.step([torch.ones(300, device="cuda"), torch.ones(5, device="cuda")])
        cut = {k: [opt.arena[k][:2 if k.endswith("scale") else 300], opt.arena[k][2:3] if k.endswith("scale") else opt.arena[k][512:517]]
               for k in keys}
        good = {k: [x.clone().view(torch.uint8).zero_().view(x.dtype) for x in parts] for k, parts in cut.items()}
        before = {k: opt.arena[k].view(torch.uint8).clone() for k in keys}
        short = [good["v"][0], good["v"][1][:4]]
        for bad in ({"v": short}, {"v": good["v"][:1]}, {"m": good["m"] + [good["m"][0]]}, {"v": good["v"] + [good["v"][1]]},
                    {"v": None}, {"v": [x.double() for x in good["v"]]}):
            with pytest.raises(ValueError):
                opt.load_state(7, **{**good, **bad})
            assert opt.step_count == 1
            for k in keys:
                assert torch.equal(opt.arena[k].view(torch.uint8), before[k]), (state, k, list(bad))
        opt.load_state(7, **good)
        assert opt.step_count == 7 and all(bool((x.float() == 0).all()) for parts in cut.values() for x in parts)


def test_gradient_scale_is_one_number():
    opt = E.AdamW([torch.zeros(8, device="cuda")])
    for n in (0, 2):
        with pytest.raises(ValueError):
            opt.step([torch.ones(8, device="cuda")], grad_scale=torch.ones(n, device="cuda"))
    assert opt.step_count == 0 and bool((opt.params[0] == 0).all())


def check_8bit_step(opt, dev, p, deq, grads, sizes, first, seed, t, scale=None):
    """One step of an 8-bit optimizer from known weights and dequantised states: bit for bit; returns the states after it."""
    after = []
    for i, n in enumerate(sizes):
        w, m, _, u = adamw32(p[i], grads[i], deq[i][0], None, deq[i][1], (*HYPER, t), True, grad_scale=scale)
        p[i] = w.to(p[i].dtype)
        assert torch.equal(dev[i].cpu(), p[i]), (t, i)
        bits = random_bits(first[i], n, seed, t)
        (qm, sm), (qu, su) = round_state(m, bits & 0xFFFF), round_state(u, bits >> 16)
        qu = torch.where((u > 0) & (qu == 0), torch.full_like(qu, 2.0 ** -9), qu)
        at, blk = opt._at[i], -(-n // 256)
        assert torch.equal(opt.arena["m"][at:at + n].cpu().float(), qm) and torch.equal(opt.arena["v"][at:at + n].cpu().float(), qu), (t, i)
        assert torch.equal(opt.arena["m_scale"][at // 256:at // 256 + blk].cpu(), sm), (t, i)
        assert torch.equal(opt.arena["v_scale"][at // 256:at // 256 + blk].cpu(), su), (t, i)
        after.append((qm * sm.repeat_interleave(256)[:n], qu * su.repeat_interleave(256)[:n]))
    return after


# Totals from 4M elements on give a warp several units (4M: two, 16M: eight), tiny and empty
# tensors between them let it pass over several tensors within its share.
LONG = [[1_400_003, 0, 1, 300, 257] + [17] * 30 + [2_600_000, 5, 0, 64] + [129, 1] * 20 + [300_001],
        [16_500_000, 33, 0, 1000]]


@pytest.mark.parametrize("sizes", LONG, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("state", ["f32", "q8"])
@pytest.mark.parametrize("types", ["plain", "mixed"])
def test_several_units_a_warp(sizes, state, types):
    """Bit for bit where a warp goes through several units and tensors: of one type
    and aligned, or of mixed types with every third tensor off its alignment."""
    g = torch.Generator().manual_seed(len(sizes))
    kinds = [(F32, BF16)] if types == "plain" else [(F32, BF16), (BF16, BF16), (F16, F32)]
    p, grads, dev, first = [], [], [], []
    for i, n in enumerate(sizes):
        pt, gt = kinds[i % len(kinds)]
        p.append(torch.randn(n, generator=g).to(pt))
        grads.append([(torch.randn(n, generator=g) * 1e-2).to(gt) for _ in range(2)])
        off = 1 if types == "mixed" and i % 3 == 0 else 0
        dev.append(torch.empty(n + off, dtype=pt, device="cuda")[off:])
        dev[-1].copy_(p[-1])
    opt = E.AdamW(dev, lr=HYPER[0], betas=HYPER[1:3], eps=HYPER[3], weight_decay=HYPER[4], state=state, seed=5)
    for i in range(len(sizes)):
        first.append(opt._at[i] + (3 << 32))    # the upper half of an element's number counts too
        opt._tensors[i].first = first[-1]
    m = [torch.zeros(n) for n in sizes]
    v = [torch.zeros(n) for n in sizes]
    deq = list(zip(m, v))
    for t in (1, 2):
        now = [gr[t - 1] for gr in grads]
        opt.step([x.cuda() for x in now])
        if state == "q8":
            deq = check_8bit_step(opt, dev, p, deq, now, sizes, first, 5, t)
            continue
        for i, n in enumerate(sizes):
            w, m[i], v[i], _ = adamw32(p[i], now[i], m[i], v[i], None, (*HYPER, t), False)
            p[i] = w.to(p[i].dtype)
            at = opt._at[i]
            assert torch.equal(dev[i].cpu(), p[i]), (t, i)
            assert torch.equal(opt.arena["m"][at:at + n].cpu(), m[i]) and torch.equal(opt.arena["v"][at:at + n].cpu(), v[i]), (t, i)
