"""Norm + gate + residual + norm, forward and backward, against 64-bit forms."""
import pytest
import torch

import sparse_ctr_embedding_gb300 as E
from dense_ref import U, act64, close, norm64, norm_size

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    E.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def make(rows, dim, st, bt, layer, gate, seed=0, offset=0.3):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = {"x": n(rows, dim).to(st), "f": (3 * n(rows, dim) + offset).to(bt), "w_post": 1 + 0.2 * n(dim), "w_pre": 1 + 0.2 * n(dim),
         "b_post": n(dim) if layer else None, "b_pre": n(dim) if layer else None,
         "dy": n(rows, dim).to(st), "dh": n(rows, dim).to(bt),
         "gate": {"none": None, "elem": n(rows, dim).to(bt), "row": n(rows, 1).to(bt), "col": n(dim)}[gate]}
    return d


def cu(d, keys):
    return {k: None if d[k] is None else d[k].cuda() for k in keys}


def d64(t):
    return None if t is None else t.detach().cpu().double()


VEC = ("w_post", "b_post", "w_pre", "b_pre")


def run_fwd(d, layer, act, rs, **kw):
    c = cu(d, ("x", "f", "gate") + VEC)
    return E.emb_norm_gate_fwd(c.pop("x"), c.pop("f"), c.pop("gate"), norm="layer" if layer else "rms", act=act, eps=1e-5,
                               res_scale=rs, **c, **kw)


def check_fwd(d, layer, act, rs, y, h, stats):
    w = {k: d64(d[k]) for k in VEC}
    a = act64(d64(d["gate"]), act)
    n = norm64(d64(d["f"]), w["w_post"], w["b_post"], layer, 1e-5)
    ref = rs * d64(d["x"]) + a * n
    size = (rs * d64(d["x"])).abs() + a.abs() * norm_size(d64(d["f"]), w["w_post"], w["b_post"], layer, 1e-5)
    close("y", y, ref, size, 40)
    y64 = d64(y)       # h is defined from y as stored
    close("h", h, norm64(y64, w["w_pre"], w["b_pre"], layer, 1e-5), norm_size(y64, w["w_pre"], w["b_pre"], layer, 1e-5), 40)
    for t, col in ((d64(d["f"]), 0), (y64, 2)):
        mean = t.mean(1) if layer else torch.zeros(t.shape[0], dtype=torch.float64)
        close("mean", stats[:, col], mean, t.abs().mean(1), 40)
        rstd = ((t - mean[:, None]).square().mean(1) + 1e-5).rsqrt()
        close("rstd", stats[:, col + 1], rstd, rstd * norm_size(t, None, None, layer, 1e-5).mean(1).clamp_min(1), 40)


TYPES = [(F32, F32), (BF16, BF16), (F16, F16), (F32, BF16), (F32, F16)]


@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (5, 8), (2, 64), (33, 72), (40, 250), (7, 256), (9, 1001), (4, 1024),
                                      (3, 1664), (2, 2047), (3, 4096), (2, 4104), (2, 8191), (2, 8192), (700, 64), (301, 520)])
@pytest.mark.parametrize("layer,gate,act", [(False, "elem", "sigmoid"), (True, "col", "sigmoid"), (True, "row", "identity"),
                                            (False, "none", "identity")])
def test_forward_sizes(rows, dim, layer, gate, act):
    st, bt = TYPES[(rows + dim) % len(TYPES)]
    d = make(rows, dim, st, bt, layer, gate, seed=dim)
    check_fwd(d, layer, act, 0.75, *run_fwd(d, layer, act, 0.75))


@pytest.mark.parametrize("st,bt", TYPES)
@pytest.mark.parametrize("dim", [96, 101])
def test_forward_types(st, bt, dim):
    for layer in (False, True):
        d = make(19, dim, st, bt, layer, "elem", seed=1)
        check_fwd(d, layer, "sigmoid", 1.0, *run_fwd(d, layer, "sigmoid", 1.0))


def test_forward_first_and_last():
    """No block yet: h = norm(x); no norm after: y alone; serving: no statistics."""
    d = make(6, 200, F32, BF16, False, "none")
    y, h, st = E.emb_norm_gate_fwd(d["x"].cuda(), None, w_pre=d["w_pre"].cuda(), eps=1e-5, block_dtype=BF16)
    assert y is None and h.dtype == BF16 and bool((st[:, :2] == 0).all())
    x64 = d64(d["x"])
    close("h", h, norm64(x64, d64(d["w_pre"]), None, False, 1e-5), norm_size(x64, d64(d["w_pre"]), None, False, 1e-5), 40)
    full = run_fwd(d, False, "identity", 1.0)[0]
    c = cu(d, ("x", "f", "w_post"))
    y, h, st = E.emb_norm_gate_fwd(c["x"], c["f"], w_post=c["w_post"], act="identity", eps=1e-5, pre=False, stats=False)
    assert h is None and st is None and torch.equal(y, full)


def test_forward_special_rows():
    """Rows of zeros and of equal values (zero variance), infinities and NaN: confined to their own row."""
    d = make(6, 128, F32, F32, True, "elem")
    base = [t.clone() for t in run_fwd(d, True, "sigmoid", 1.0)]
    d["f"][0] = 0.0
    d["f"][1] = 5.0
    d["f"][2, 7] = float("inf")
    d["f"][3, 9] = float("nan")
    d["gate"][4, :2] = torch.tensor([float("inf"), -float("inf")])
    y, h, st = run_fwd(d, True, "sigmoid", 1.0)
    for t, b in ((y, base[0]), (h, base[1]), (st, base[2])):
        assert torch.equal(t[5], b[5])
    assert bool(torch.isfinite(y[:2]).all()) and bool(torch.isfinite(y[4]).all())
    want = d["x"][:2].double() + act64(d["gate"][:2].double(), "sigmoid") * d["b_post"].double()   # the norm of a constant is 0
    close("y of constant rows", y[:2], want, 1 + want.abs(), 40)
    assert bool(torch.isnan(y[2, 7]) & torch.isnan(h[2]).all() & torch.isnan(y[3]).all())
    big = make(2, 64, F32, F32, False, "none")
    big["f"] = big["f"] * 1e18       # squares of 1e37: still finite sums
    close("y of large rows", run_fwd(big, False, "identity", 1.0)[0], *(lambda n: (big["x"].double() + n, big["x"].double().abs() + n.abs()))(
        norm64(big["f"].double(), big["w_post"].double(), None, False, 1e-5)), 40)


def grads64(d, y, layer, act, rs, has_f=True, has_dh=True, has_dy=True):
    """The formulas in 64 bits at the stored y, and the size of the terms behind each gradient."""
    eps = 1e-5
    w = {k: d64(d[k]) for k in VEC}
    one = torch.ones(y.shape[1], dtype=torch.float64)
    zero = torch.zeros_like(d64(y))

    def hat(t):
        c = t - t.mean(1, keepdim=True) if layer else t
        r = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
        return c * r, r, norm_size(t, None, None, layer, eps)

    m = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    out, size = {}, {}
    dt, s_dt = (d64(d["dy"]), d64(d["dy"]).abs()) if has_dy else (zero, zero)
    if has_dh:
        yh, r, s_yh = hat(d64(y))
        dh = d64(d["dh"])
        e = dh * (one if w["w_pre"] is None else w["w_pre"])
        dt = dt + r * (e - yh * m(e * yh) - (m(e) if layer else 0))
        s_dt = s_dt + r * (e.abs() + s_yh * m(e.abs() * s_yh) + (m(e.abs()) if layer else 0)) * m(s_yh).clamp_min(1)
        out["dw_pre"], size["dw_pre"] = (dh * yh).sum(0), (dh.abs() * s_yh).sum(0)
        out["db_pre"], size["db_pre"] = dh.sum(0), dh.abs().sum(0)
    if not has_f:
        return {**out, "dx": dt}, {**size, "dx": s_dt}
    out["dx"], size["dx"] = rs * dt, abs(rs) * s_dt
    fh, r, s_fh = hat(d64(d["f"]))
    wp = one if w["w_post"] is None else w["w_post"]
    n = fh * wp + (0 if w["b_post"] is None else w["b_post"])
    s_n = s_fh * wp.abs() + (0 if w["b_post"] is None else w["b_post"].abs())
    a = act64(d64(d["gate"]), act)
    slope = a * (1 - a) if act == "sigmoid" else torch.ones_like(a)
    dg, s_dg = dt * n * slope, s_dt * s_n
    if d["gate"] is not None:
        g = d["gate"]
        if g.dim() == 1:
            out["dgate"], size["dgate"] = dg.sum(0), s_dg.sum(0)
        elif g.shape[1] == 1 and y.shape[1] != 1:
            out["dgate"], size["dgate"] = dg.sum(1, keepdim=True), s_dg.sum(1, keepdim=True)
        else:
            out["dgate"], size["dgate"] = dg, s_dg
    dn, s_dn = dt * a, s_dt * a.abs()
    out["dw_post"], size["dw_post"] = (dn * fh).sum(0), (s_dn * s_fh).sum(0)
    out["db_post"], size["db_post"] = dn.sum(0), s_dn.sum(0)
    e, s_e = dn * wp, s_dn * wp.abs()
    out["df"] = r * (e - fh * m(e * fh) - (m(e) if layer else 0))
    size["df"] = r * (s_e + s_fh * m(s_e * s_fh) + (m(s_e) if layer else 0)) * m(s_fh).clamp_min(1)
    return out, size


def run_bwd(d, y, stats, layer, act, rs, **kw):
    c = cu(d, ("dy", "dh", "f", "gate") + VEC)
    return E.emb_norm_gate_bwd(c.pop("dy"), c.pop("dh"), y, c.pop("f"), c.pop("gate"), stats, norm="layer" if layer else "rms",
                               act=act, eps=1e-5, res_scale=rs, **c, **kw)


def check_bwd(d, y, got, layer, act, rs, **has):
    ref, size = grads64(d, y, layer, act, rs, **has)
    rows = y.shape[0]
    for k, v in got.items():
        if v is None:
            continue
        over_rows = k[:2] in ("dw", "db") or (k == "dgate" and d["gate"].dim() == 1)
        close(k, v, ref[k].reshape(v.shape), size[k].reshape(v.shape), rows + 128 if over_rows else 128)


@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (5, 8), (2, 64), (33, 72), (40, 250), (7, 256), (9, 1001), (4, 1024),
                                      (3, 1664), (2, 2047), (3, 4096), (2, 4104), (2, 8191), (3, 8192), (700, 64), (301, 520),
                                      (5000, 24), (1300, 1024), (400, 8192)])
@pytest.mark.parametrize("layer,gate,act", [(False, "elem", "sigmoid"), (True, "col", "sigmoid"), (True, "row", "identity"),
                                            (False, "none", "identity")])
def test_backward_sizes(rows, dim, layer, gate, act):
    st, bt = TYPES[(rows + dim) % len(TYPES)]
    d = make(rows, dim, st, bt, layer, gate, seed=dim + 1)
    y, _, stats = run_fwd(d, layer, act, 0.75)
    got = run_bwd(d, y, stats, layer, act, 0.75)
    check_bwd(d, y, got, layer, act, 0.75)
    again = run_bwd(d, y, stats, layer, act, 0.75)
    assert all(torch.equal(v, again[k]) for k, v in got.items() if v is not None)


@pytest.mark.parametrize("st,bt", TYPES)
@pytest.mark.parametrize("dim", [96, 101])
def test_backward_types(st, bt, dim):
    for gate in ("elem", "row", "col"):
        d = make(19, dim, st, bt, True, gate, seed=2)
        y, _, stats = run_fwd(d, True, "sigmoid", 1.0)
        check_bwd(d, y, run_bwd(d, y, stats, True, "sigmoid", 1.0), True, "sigmoid", 1.0)


@pytest.mark.parametrize("has", [dict(has_f=False), dict(has_dh=False), dict(has_dy=False), dict(has_f=False, has_dy=False)])
def test_backward_absent_parts(has):
    d = make(37, 136, F32, F32, True, "none", seed=3)
    y, _, stats = run_fwd(d, True, "identity", 0.5)
    if not has.get("has_f", True):
        _, _, stats = E.emb_norm_gate_fwd(y, None, w_pre=d["w_pre"].cuda(), b_pre=d["b_pre"].cuda(), norm="layer", eps=1e-5)
        d.update(f=None, w_post=None, b_post=None)
    for k, names in (("has_dh", ("dh", "w_pre", "b_pre")), ("has_dy", ("dy",))):
        if not has.get(k, True):
            d.update({n: None for n in names})
    check_bwd(d, y, run_bwd(d, y, stats, True, "identity", 0.5), True, "identity", 0.5, **has)


def test_backward_of_no_rows_gives_zero_sums():
    d = make(0, 40, F32, F32, True, "col")
    y, h, stats = run_fwd(d, True, "sigmoid", 1.0)
    assert y.shape == h.shape == (0, 40)
    got = run_bwd(d, y, stats, True, "sigmoid", 1.0)
    for k in ("dw_post", "db_post", "dw_pre", "db_pre", "dgate"):
        assert got[k].shape == (40,) and bool((got[k] == 0).all())


@pytest.mark.parametrize("layer,gate", [(False, "elem"), (True, "col"), (True, "row")])
def test_gradients_against_differences(layer, gate):
    """<gradient, v> for random directions v against central differences of the
    64-bit definition (step 1e-5: the differences are good to about 1e-9)."""
    rows, dim, rs, eps = 13, 88, 0.6, 1e-5
    d = make(rows, dim, F32, F32, layer, gate, seed=5)
    y, _, stats = run_fwd(d, layer, "sigmoid", rs)
    got = run_bwd(d, y, stats, layer, "sigmoid", rs)
    _, size = grads64(d, y, layer, "sigmoid", rs)
    # dy and dh reach y directly; the branch and the residual reach it through dt = dx / rs
    p = {k: d64(d[k]) for k in ("x", "f", "gate") + VEC}
    y64, dy, dh = d64(y), d64(d["dy"]), d64(d["dh"])

    def loss(q, shift):
        """The step's loss, its y moved from the stored one by what the inputs move it."""
        n = lambda z: norm64(z["f"], z["w_post"], z["b_post"], layer, eps) * act64(z["gate"], "sigmoid") + rs * z["x"]  # noqa: E731
        yy = y64 + (n(q) - n(p))
        return (dy * yy).sum() + (dh * norm64(yy, q["w_pre"], q["b_pre"], layer, eps)).sum()

    g = torch.Generator().manual_seed(9)
    names = {"x": "dx", "f": "df", "gate": "dgate", **{k: "d" + k for k in VEC}}
    for k, name in names.items():
        if p[k] is None:
            continue
        v = torch.randn(p[k].shape, generator=g, dtype=torch.float64)
        up, down = dict(p), dict(p)
        up[k], down[k] = p[k] + 1e-5 * v, p[k] - 1e-5 * v
        slope = float((loss(up, 1) - loss(down, -1)) / 2e-5)
        mine = float((d64(got[name]) * v).sum())
        bound = float((size[name].reshape(v.shape) * v.abs()).sum()) * (rows + 128) * U + 1e-6 * abs(slope) + 1e-6
        assert abs(mine - slope) <= bound, (name, mine, slope, bound)


def test_unaligned_views_and_another_stream():
    """Rows that start off 16-byte boundaries take the element-wise path; work on a side stream is ordered there."""
    d = make(50, 264, F32, BF16, False, "elem", seed=8)
    want = run_fwd(d, False, "sigmoid", 1.0)
    buf = torch.zeros(50 * 264 + 1, dtype=BF16, device="cuda")
    f = buf[1:].view(50, 264)
    f.copy_(d["f"])
    s = torch.cuda.Stream()
    c = cu(d, ("x", "gate", "w_post", "w_pre"))
    s.wait_stream(torch.cuda.current_stream())
    got = E.emb_norm_gate_fwd(c["x"], f, c["gate"], w_post=c["w_post"], w_pre=c["w_pre"], eps=1e-5, stream=s)
    s.synchronize()
    check_fwd(d, False, "sigmoid", 1.0, *got)
    y, h, st = want
    g1 = run_bwd(d, y, st, False, "sigmoid", 1.0)
    g2 = E.emb_norm_gate_bwd(d["dy"].cuda(), d["dh"].cuda(), y, f, c["gate"], st, w_post=c["w_post"], w_pre=c["w_pre"], eps=1e-5)
    check_bwd(d, y, g1, False, "sigmoid", 1.0)
    check_bwd(d, y, g2, False, "sigmoid", 1.0)


@pytest.mark.parametrize("st,bt", [(F32, F32), (F32, BF16)])
@pytest.mark.parametrize("kind", ["elem", "row", "col"])
@pytest.mark.parametrize("dim,full", [(64, False), (64, True), (4, False), (8192, False)])
def test_sigmoid_of_float32_rows(st, bt, kind, dim, full):
    """With x = 0 and f = 1 (whose norm is exactly 1 here) y is the sigmoid itself.
    Where rows are float32 it is good to 12 u over the whole range of gates: the
    power of two 4 u, its correction, the sum and y's product 1 u each, the
    reciprocal 2 u.  The gate's gradient a (1 - a) has a's error twice, and for
    a near 1 what 1 - a cancels."""
    g = torch.Generator().manual_seed(dim)
    top = 87.0                       # below, the sigmoid leaves the normal range
    gates = torch.cat([torch.linspace(-top, top, 700), torch.randn(300, generator=g) * 4, torch.tensor([0.0, -0.0, top, -top])])
    gates = gates.to(bt)
    if kind == "col":
        gate = gates.float()[torch.arange(dim) % gates.numel()]
        rows, all_gates = 3, gate.expand(3, dim)
    else:
        rows = gates.numel()
        gate = gates[:, None] if kind == "row" else gates[(torch.arange(rows)[:, None] + torch.arange(dim)) % rows]
        all_gates = gate.expand(rows, dim)
    x, f, one = torch.zeros(rows, dim, dtype=st).cuda(), torch.ones(rows, dim, dtype=bt).cuda(), torch.ones(dim).cuda()
    kw = dict(w_post=one, w_pre=one, eps=1e-30) if full else dict(w_post=one, eps=1e-30, pre=False)
    y, h, stats = E.emb_norm_gate_fwd(x, f, gate.cuda(), **kw)
    assert bool((stats[:, 1] == 1).all())
    a = 1 / (1 + torch.exp(-all_gates.double()))
    err = (y.cpu().double() - a).abs()
    assert bool((err <= 12 * U * a + 2.0 ** -126).all()), float((err / a).max() / U)
    if bt != F32 and kind != "col":
        return                        # the gradient is rounded to the gate's type
    dy = torch.zeros(rows, dim)       # one row at a time in the sums over rows, one column in those over columns
    dy[torch.arange(rows), torch.arange(rows) % dim] = 1.0
    got = E.emb_norm_gate_bwd(dy.cuda(), None, y, f, gate.cuda(), stats, w_post=one, eps=1e-30)["dgate"].cpu().double()
    slope = torch.where(dy != 0, a * (1 - a), torch.zeros_like(a))
    want = slope.sum(1, keepdim=True) if kind == "row" else slope.sum(0) if kind == "col" else slope
    of = torch.where(dy != 0, a, torch.zeros_like(a))
    size = of.sum(1, keepdim=True) if kind == "row" else of.sum(0) if kind == "col" else of
    err = (got.reshape(want.shape) - want).abs()
    assert bool((err <= 12 * U * want + 5 * U * size + 2.0 ** -126).all())


@pytest.mark.parametrize("st,bt", [(F32, F32), (F32, F16), (BF16, BF16)])
def test_sigmoid_of_gates_out_of_range(st, bt):
    """Gates of any size and NaN: 0, 1 or NaN, nothing else in the row touched."""
    gate = torch.zeros(7, 64, dtype=bt)
    values = torch.tensor([200.0, -200.0, 65504.0, -65504.0, float("inf"), -float("inf"), float("nan")]).to(bt)
    gate[:, 5] = values
    x, f, one = torch.zeros(7, 64, dtype=st).cuda(), torch.ones(7, 64, dtype=bt).cuda(), torch.ones(64).cuda()
    y = E.emb_norm_gate_fwd(x, f, gate.cuda(), w_post=one, eps=1e-30, pre=False)[0].cpu().float()
    assert y[:6, 5].tolist() == [1.0, 0.0, 1.0, 0.0, 1.0, 0.0] and bool(torch.isnan(y[6, 5]))
    y[:, 5] = 0.5
    assert bool((y == 0.5).all())


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("gate", ["elem", "row", "col"])
@pytest.mark.parametrize("rows,dim", [(40_000, 64), (5000, 1001), (3000, 2048), (2000, 1100)])
def test_forward_of_many_rows_a_team(rows, dim, gate, layer):
    """Several rows to each team, the next one loaded while one is reduced: y, h and the statistics of every row."""
    st, bt = TYPES[(dim + layer) % len(TYPES)]
    d = make(rows, dim, st, bt, layer, gate, seed=dim)
    check_fwd(d, layer, "sigmoid", 0.75, *run_fwd(d, layer, "sigmoid", 0.75))


@pytest.mark.parametrize("st,bt", [(F32, F32), (BF16, BF16), (F32, F16)])
@pytest.mark.parametrize("dim", [1100, 2047, 4096, 8191, 8192])
def test_layer_norm_with_gates_in_large_teams(dim, st, bt):
    """Every array there, layer norms, a gate per element, teams of 512 and 1024 threads: forward and backward."""
    d = make(400, dim, st, bt, True, "elem", seed=dim)
    y, h, stats = run_fwd(d, True, "sigmoid", 0.75)
    check_fwd(d, True, "sigmoid", 0.75, y, h, stats)
    check_bwd(d, y, run_bwd(d, y, stats, True, "sigmoid", 0.75), True, "sigmoid", 0.75)
