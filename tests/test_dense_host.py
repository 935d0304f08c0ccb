"""Refusals of the dense-tower operators: host checks, made before any CUDA call
(pointers here are plain numbers that nothing reads), and the binding's."""
import ctypes

import pytest
import torch

import sparse_ctr_embedding_gb300 as E

P = 1 << 20     # an aligned address; never dereferenced by a refused call


@pytest.fixture(scope="module", autouse=True)
def built():
    E.build()


def refused(rc, name="EMB_ERR_INVALID_ARG"):
    assert E.STATUS[rc] == name, E.emb_last_error()
    assert E.emb_last_error()


def quant(**kw):
    a = dict(x=P, t=0, rows=100, cols=200, ldx=200, br=1, q=P, ldq=208, s=P, qt=None, ldqt=0, st=None)
    a.update(kw)
    return E.lib().emb_fp8_quantize(a["x"], a["t"], a["rows"], a["cols"], a["ldx"], a["br"], a["q"], a["ldq"], a["s"], a["qt"],
                                    a["ldqt"], a["st"], None)


@pytest.mark.parametrize("kw", [dict(t=3), dict(rows=-1), dict(cols=-1), dict(br=2), dict(q=None), dict(s=None), dict(qt=P, ldqt=112),
                                dict(ldx=199), dict(ldq=200), dict(ldq=192), dict(q=P + 8), dict(x=P + 2), dict(x=None), dict(s=P + 2),
                                dict(qt=P, st=P, ldqt=96)], ids=str)
def test_quantize_refuses(kw):
    refused(quant(**kw))


def test_quantize_too_many_tiles_and_empty():
    refused(quant(rows=1 << 40, cols=1 << 20, ldx=1 << 20, ldq=1 << 20), "EMB_ERR_UNSUPPORTED")
    assert quant(rows=0) == 0 and quant(cols=0, ldx=0, ldq=0) == 0


def matmul(**kw):
    m, n, k = kw.pop("mnk", (40, 50, 200))
    a = dict(a=P, lda=208, sa=P, ar=1, b=P, ldb=208, sb=P, br=128, bias=None, out=P, t=0, ldo=n, ws=P, wsb=1 << 40)
    a.update(kw)
    return E.lib().emb_fp8_matmul(a["a"], a["lda"], a["sa"], a["ar"], a["b"], a["ldb"], a["sb"], a["br"], m, n, k, a["bias"], a["out"],
                                  a["t"], a["ldo"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw", [dict(mnk=(-1, 2, 3)), dict(t=5), dict(ar=64), dict(br=0), dict(lda=200), dict(ldb=192), dict(ldo=49),
                                dict(a=None), dict(b=None), dict(sa=None), dict(sb=None), dict(out=None), dict(a=P + 8), dict(b=P + 1),
                                dict(out=P + 2), dict(bias=P + 1)], ids=str)
def test_matmul_refuses(kw):
    refused(matmul(**kw))


def test_matmul_limits():
    refused(matmul(mnk=(1 << 31, 8, 16)), "EMB_ERR_UNSUPPORTED")
    assert matmul(mnk=(0, 50, 200)) == 0
    with pytest.raises(E.EmbError) as ei:
        E.emb_fp8_matmul_workspace_size(4, -1, 4)
    assert ei.value.name == "EMB_ERR_INVALID_ARG"


def norm_desc(**kw):
    a = dict(rows=4, dim=64, st=0, bt=0, norm=0, gate=0, act=0, eps=1e-6, rs=1.0)
    a.update(kw)
    return E._NormGate(a["rows"], a["dim"], a["st"], a["bt"], a["norm"], a["gate"], a["act"], a["eps"], a["rs"])


def fwd(ptrs=(), **kw):
    a = dict(x=P, f=P, gate=None, wp=None, bp=None, wq=None, bq=None, y=P, h=P, stats=P)
    a.update(ptrs)
    d = norm_desc(**kw)
    return E.lib().emb_norm_gate_fwd(ctypes.byref(d), *[a[k] for k in ("x", "f", "gate", "wp", "bp", "wq", "bq", "y", "h", "stats")], None)


def bwd(ptrs=(), **kw):
    a = dict(dy=P, dh=P, y=P, f=P, gate=None, stats=P, wp=None, bp=None, wq=None, dx=P, df=P, dg=None, dwp=None, dbp=None, dwq=None,
             dbq=None, ws=P, wsb=1 << 40)
    a.update(ptrs)
    d = norm_desc(**kw)
    return E.lib().emb_norm_gate_bwd(ctypes.byref(d), *[a[k] for k in ("dy", "dh", "y", "f", "gate", "stats", "wp", "bp", "wq", "dx", "df",
                                                                        "dg", "dwp", "dbp", "dwq", "dbq", "ws", "wsb")], None)


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(dim=0), dict(st=1, bt=2), dict(bt=3), dict(norm=2), dict(gate=4), dict(act=2),
                                dict(eps=0.0), dict(eps=float("nan")), dict(rs=float("inf"))], ids=str)
def test_norm_refuses_bad_descriptions(kw):
    refused(fwd(**kw))
    refused(bwd(**kw))


def test_norm_refuses_bad_arrays():
    refused(fwd(dim=8193), "EMB_ERR_UNSUPPORTED")
    for ptrs, kw in [(dict(x=None), {}), (dict(y=None), {}), (dict(f=None), {}), (dict(f=None, y=None, h=None), {}),
                     (dict(gate=P), {}), ({}, dict(gate=1)), (dict(bp=P), {}), (dict(bq=P), {}), (dict(h=None, wq=P), {}),
                     (dict(x=P + 2), {}), (dict(stats=P + 8), {}), (dict(f=None, y=None, wp=P), {}), (dict(gate=P + 2), dict(gate=3))]:
        refused(fwd(ptrs, **kw))
    for ptrs, kw in [(dict(dy=None, dh=None), {}), (dict(stats=None), {}), (dict(y=None), {}), (dict(dh=None, wq=P), {}),
                     (dict(dh=None, dwq=P), {}), (dict(f=None), {}), (dict(gate=P), {}), (dict(dg=P), {}), ({}, dict(gate=2)),
                     (dict(dbp=P), {}), (dict(dwp=P + 2), {}), (dict(dy=P + 1), {}), (dict(stats=P + 4), {})]:
        refused(bwd(ptrs, **kw))
    refused(bwd(dict(dwp=P, ws=None)), "EMB_ERR_WORKSPACE")
    refused(bwd(dict(dwp=P, wsb=4)), "EMB_ERR_WORKSPACE")
    refused(bwd(dict(dwp=P, ws=P + 4)), "EMB_ERR_WORKSPACE")
    assert fwd(rows=0) == 0


def adamw(tensor=(), grads=P, n=1, **kw):
    a = dict(lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, step=1, state=0)
    a.update(kw)
    t = dict(param=P, copy=None, m=P, v=P, ms=None, vs=None, n=10, first=0, pt=0, gt=0, ct=1)
    t.update(tensor)
    arr = (E._AdamwTensor * 1)(E._AdamwTensor(*[t[k] for k in ("param", "copy", "m", "v", "ms", "vs", "n", "first", "pt", "gt", "ct")]))
    g = (ctypes.c_void_p * 1)(grads)
    p = E._AdamwParams(a["lr"], a["b1"], a["b2"], a["eps"], a["wd"], a["step"], a["state"], 0, None)
    return E.lib().emb_adamw_step(arr, g, n, ctypes.byref(p), None)


@pytest.mark.parametrize("kw", [dict(lr=-1.0), dict(lr=float("nan")), dict(b1=1.0), dict(b2=-0.1), dict(eps=0.0), dict(eps=1e-60),
                                dict(wd=-1.0), dict(step=0), dict(state=2), dict(n=-1), dict(state=1), dict(grads=None), dict(grads=P + 2),
                                dict(tensor=dict(n=-1)), dict(tensor=dict(first=-1)), dict(tensor=dict(pt=3)), dict(tensor=dict(gt=-1)),
                                dict(tensor=dict(param=None)), dict(tensor=dict(m=None)), dict(tensor=dict(v=P + 2)),
                                dict(tensor=dict(copy=P, pt=1)), dict(tensor=dict(copy=P, ct=0)), dict(tensor=dict(copy=P + 1))], ids=str)
def test_adamw_refuses(kw):
    refused(adamw(**kw))


def test_adamw_of_nothing():
    assert adamw(n=0) == 0
    assert adamw(tensor=dict(n=0, param=None, m=None, v=None), grads=None) == 0


def test_binding_refuses_host_tensors_and_bad_shapes():
    with pytest.raises(ValueError):
        E.emb_fp8_quantize(torch.zeros(4, 4))
    with pytest.raises(ValueError):
        E.emb_fp8_matmul(torch.zeros(4, 16).to(torch.float8_e4m3fn), torch.ones(1, 4), torch.zeros(4, 16).to(torch.float8_e4m3fn),
                         torch.ones(1, 4))
    x = torch.zeros(4, 6)
    for gate in (torch.zeros(4), torch.zeros(1, 6), torch.zeros(6, dtype=torch.float16), torch.zeros(4, 5)):
        with pytest.raises((ValueError, TypeError)):
            E.emb_norm_gate_fwd(x, x, gate, stream=0)
    with pytest.raises(ValueError):
        E.emb_norm_gate_fwd(x, torch.zeros(4, 7), stream=0)
    with pytest.raises(ValueError):
        E.emb_norm_gate_bwd(None, None, x, None, None, torch.zeros(4, 4), stream=0)


def test_constants_match_the_header():
    import re
    text = open(E.HEADER).read()
    for name in ("EMB_FLAG_OP_TIMEOUT", "EMB_FP8_BLOCK", "EMB_ADAM_BLOCK", "EMB_NORM_MAX_DIM"):
        assert int(re.search(rf"^#define {name}\s+(\d+)", text, re.M).group(1)) == getattr(E, name)


def test_lost_waits_are_refused_out_of_range():
    for role, step in ((-2, 0), (4, 0), (0, -1), (0, 1 << 31)):
        refused(E.lib().emb_debug_lose_op_wait(role, step))
    with pytest.raises(ValueError):
        E.emb_debug_lose_op_wait("store")
    E.emb_debug_lose_op_wait(None)


class OnDevice(torch.Tensor):
    """A host tensor that says it is on GPU `where`: for the checks that come before any launch."""

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        if func == torch.Tensor.get_device:
            return args[0].where
        if func == torch.Tensor.is_cuda.__get__:
            return True
        return super().__torch_function__(func, types, args, kwargs or {})


def on(where, t):
    t = t.as_subclass(OnDevice)
    t.where = where
    return t


class NoLaunch:
    """The library without its launches."""

    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        def launched(*args):
            raise AssertionError(name + " was called")
        return getattr(self.lib, name) if name.endswith("workspace_size") else launched


F8 = torch.float8_e4m3fn


def calls(where):
    """Each operator with its tensors on the GPUs that `where` names (default 0)."""
    w = lambda k, t: on(where.get(k, 0), t)  # noqa: E731
    z = lambda *s: torch.zeros(*s)  # noqa: E731
    vec = lambda: {k: w(k, z(6)) for k in ("w_post", "b_post", "w_pre", "b_pre")}  # noqa: E731
    return {
        "quantize": lambda: E.emb_fp8_quantize(w("x", z(4, 6))),
        "matmul": lambda: E.emb_fp8_matmul(w("a", z(4, 16).to(F8)), w("sa", z(1, 4)), w("b", z(8, 16).to(F8)), w("sb", z(1, 8)), bias=w("bias", z(8)),
                                           out=w("out", z(4, 8)), workspace=w("workspace", z(64))),
        "fwd": lambda: E.emb_norm_gate_fwd(w("x", z(4, 6)), w("f", z(4, 6)), w("gate", z(4, 6)), norm="layer", **vec()),
        "bwd": lambda: E.emb_norm_gate_bwd(w("dy", z(4, 6)), w("dh", z(4, 6)), w("y", z(4, 6)), w("f", z(4, 6)), w("gate", z(4, 6)),
                                           w("stats", z(4, 4)), norm="layer", workspace=w("workspace", z(4000)), **vec()),
    }


@pytest.mark.parametrize("op,names", [("quantize", "x"), ("matmul", "a sa b sb bias out workspace"), ("fwd", "x f gate w_post b_post w_pre b_pre"),
                                      ("bwd", "dy dh y f gate stats w_post b_post w_pre b_pre workspace")])
def test_operands_on_another_device_are_refused(monkeypatch, op, names):
    """One operand on another GPU, or all on one that is not current: refused before anything is launched."""
    stub = NoLaunch(E.lib())
    monkeypatch.setattr(E, "lib", lambda: stub)
    monkeypatch.setattr(E, "_current_device", lambda: 0)
    monkeypatch.setattr(E, "_raw_stream", lambda stream, dev=None: 0)
    with pytest.raises(AssertionError, match="was called"):
        calls({})[op]()                      # all on the current device: it would have been launched
    for name in names.split():
        with pytest.raises(ValueError, match="cuda:"):
            calls({name: 1})[op]()
    monkeypatch.setattr(E, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="cuda:1"):
        calls({})[op]()
    with pytest.raises(AssertionError, match="was called"):
        calls({n: 1 for n in names.split()})[op]()


def test_plan_of_a_product():
    refused(E.lib().emb_debug_fp8_matmul_plan(4, 4, 4, None))
    refused(E.lib().emb_debug_fp8_matmul_plan(4, -1, 4, (ctypes.c_int64 * 4)()))
    assert E.emb_debug_fp8_matmul_plan(1, 100, 300)[0] == 0
    cols, tiles, blocks, steps = E.emb_debug_fp8_matmul_plan(1000, 300, 500)
    assert cols in (64, 128, 256) and tiles == 8 * -(-300 // cols) and blocks >= 1 and steps >= 0


class Reads:
    """The library as far as a product, which reads rows of codes as its kernels do: in whole 16 bytes."""

    def __init__(self, lib, short):
        self.lib, self.short, self.rows = lib, short.data_ptr(), []

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return getattr(self.lib, name)

        def product(a, lda, sa, ar, b, ldb, sb, br, m, n, k, *_):
            for at, ld, rows in ((a, lda, m), (b, ldb, n)):
                assert at != self.short, "reads past the end of a tensor"
                assert ld % 16 == 0
                self.rows.append([ctypes.string_at(at + i * ld, -(-k // 16) * 16)[:k] for i in range(rows)])
            return 0
        return product


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("k", [1, 15, 20, 500])
def test_rows_are_not_read_past_their_storage(monkeypatch, rows, k):
    """Codes whose storage ends with the last row's last byte are laid out anew; others are taken as they are."""
    ld = -(-k // 16) * 16
    g = torch.Generator().manual_seed(k)
    short = torch.randint(0, 127, ((rows - 1) * ld + k,), dtype=torch.uint8, generator=g).view(F8).as_strided((rows, k), (ld, 1))
    room = torch.randint(0, 127, (5, ld), dtype=torch.uint8, generator=g).view(F8)[:, :k]
    stub = Reads(E.lib(), short)
    monkeypatch.setattr(E, "lib", lambda: stub)
    monkeypatch.setattr(E, "_current_device", lambda: 0)
    monkeypatch.setattr(E, "_raw_stream", lambda stream, dev=None: 0)
    for a, b in ((short, room), (room, short)):
        E.emb_fp8_matmul(on(0, a), on(0, torch.zeros(-(-k // 128), a.shape[0])), on(0, b), on(0, torch.zeros(-(-k // 128), b.shape[0])),
                         out=on(0, torch.zeros(a.shape[0], b.shape[0])))
    want = [bytes(r.tolist()) for r in short.contiguous().view(torch.uint8)]
    assert stub.rows[0] == stub.rows[3] == want and stub.rows[1] == stub.rows[2]
