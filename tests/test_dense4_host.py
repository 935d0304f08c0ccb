"""Refusals of the 4-bit operators, Muon and the plain embeddings: host checks, made
before any CUDA call (pointers here are plain numbers that nothing reads), and the binding's."""
import ctypes
import re

import pytest
import torch

import sparse_ctr_embedding_gb300 as E
from test_dense_host import NoLaunch, on, refused

P = 1 << 20     # an aligned address; never dereferenced by a refused call


@pytest.fixture(scope="module", autouse=True)
def built():
    E.build()


def quant(**kw):
    a = dict(x=P, t=0, rows=100, cols=200, ldx=200, br=1, q=P, ldq=112, s=P, qt=None, ldqt=0, st=None)
    a.update(kw)
    return E.lib().emb_fp4_quantize(*[a[k] for k in ("x", "t", "rows", "cols", "ldx", "br", "q", "ldq", "s", "qt", "ldqt", "st")], None)


@pytest.mark.parametrize("kw", [dict(t=3), dict(rows=-1), dict(cols=-1), dict(br=2), dict(br=128), dict(q=None), dict(s=None),
                                dict(qt=P, ldqt=64), dict(ldx=199), dict(ldq=100), dict(ldq=96), dict(q=P + 8), dict(x=P + 2),
                                dict(x=None), dict(qt=P, st=P, ldqt=48), dict(qt=P, st=P, ldqt=56), dict(qt=P + 4, st=P, ldqt=64)], ids=str)
def test_quantize_refuses(kw):
    refused(quant(**kw))


def test_quantize_limits_and_empty():
    refused(quant(rows=1 << 30, cols=1 << 20, ldx=1 << 20, ldq=1 << 20), "EMB_ERR_UNSUPPORTED")
    refused(quant(rows=1 << 31, cols=8, ldx=8, ldq=16), "EMB_ERR_UNSUPPORTED")
    assert quant(rows=0) == 0 and quant(cols=0, ldx=0, ldq=0) == 0


def back(**kw):
    a = dict(q=P, ldq=112, s=P, rows=100, cols=200, out=P, t=1, ldo=200)
    a.update(kw)
    return E.lib().emb_fp4_dequantize(*[a[k] for k in ("q", "ldq", "s", "rows", "cols", "out", "t", "ldo")], None)


@pytest.mark.parametrize("kw", [dict(t=-1), dict(rows=-1), dict(cols=-5), dict(q=None), dict(s=None), dict(out=None), dict(ldq=96), dict(ldq=104),
                                dict(q=P + 8), dict(ldo=199), dict(out=P + 1)], ids=str)
def test_dequantize_refuses(kw):
    refused(back(**kw))


def test_dequantize_limits_and_empty():
    refused(back(rows=1 << 31, cols=8, ldo=8, ldq=16), "EMB_ERR_UNSUPPORTED")
    assert back(rows=0) == 0 and back(cols=0) == 0


def matmul(**kw):
    m, n, k = kw.pop("mnk", (40, 50, 200))
    a = dict(a=P, lda=112, sa=P, b=P, ldb=112, sb=P, bias=None, out=P, t=0, ldo=n, ws=P, wsb=1 << 40)
    a.update(kw)
    return E.lib().emb_fp4_matmul(a["a"], a["lda"], a["sa"], a["b"], a["ldb"], a["sb"], m, n, k, a["bias"], a["out"], a["t"], a["ldo"],
                                  a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw", [dict(mnk=(-1, 2, 3)), dict(t=5), dict(lda=100), dict(ldb=96), dict(ldo=49), dict(a=None), dict(b=None),
                                dict(sa=None), dict(sb=None), dict(out=None), dict(a=P + 8), dict(b=P + 1), dict(sa=P + 8), dict(sb=P + 4),
                                dict(out=P + 2), dict(bias=P + 1)], ids=str)
def test_matmul_refuses(kw):
    refused(matmul(**kw))


def test_matmul_limits():
    refused(matmul(mnk=(1 << 31, 8, 16)), "EMB_ERR_UNSUPPORTED")
    refused(matmul(lda=1 << 39), "EMB_ERR_UNSUPPORTED")
    assert matmul(mnk=(0, 50, 200)) == 0 and matmul(mnk=(40, 0, 200)) == 0
    with pytest.raises(E.EmbError) as ei:
        E.emb_fp4_matmul_workspace_size(4, -1, 4)
    assert ei.value.name == "EMB_ERR_INVALID_ARG"
    refused(E.lib().emb_fp4_matmul_workspace_size(1, 1, 1, None))
    refused(E.lib().emb_debug_fp4_matmul_plan(4, 4, 4, None))
    refused(E.lib().emb_debug_fp4_matmul_plan(4, -1, 4, (ctypes.c_int64 * 5)()))
    assert E.emb_debug_fp4_matmul_plan(1, 100, 300)[0] == 0


def muon(tensor=(), grads=P, n=1, ws=P, wsb=1 << 40, **kw):
    t = dict(p=P, m=P, rows=10, cols=20, pt=0, gt=0, scale=1.0)
    t.update(tensor)
    a = dict(lr=1e-3, mom=0.9, wd=0.0, nesterov=1, products=0, gs=None)
    a.update(kw)
    arr = (E._MuonTensor * 1)(E._MuonTensor(*[t[k] for k in ("p", "m", "rows", "cols", "pt", "gt", "scale")]))
    g = (ctypes.c_void_p * 1)(grads)
    o = E._MuonParams(*[a[k] for k in ("lr", "mom", "wd", "nesterov", "products", "gs")])
    return E.lib().emb_muon_step(arr, g, n, ctypes.byref(o), ws, wsb, None)


@pytest.mark.parametrize("kw", [dict(lr=-1.0), dict(lr=float("nan")), dict(mom=1.0), dict(mom=-0.1), dict(mom=float("nan")), dict(wd=-1.0),
                                dict(products=2), dict(n=-1), dict(grads=None), dict(grads=P + 2), dict(gs=P + 1), dict(tensor=dict(rows=-1)),
                                dict(tensor=dict(cols=-1)), dict(tensor=dict(pt=3)), dict(tensor=dict(gt=-1)), dict(tensor=dict(p=None)),
                                dict(tensor=dict(m=None)), dict(tensor=dict(m=P + 2)), dict(tensor=dict(p=P + 2)),
                                dict(tensor=dict(scale=float("inf"))), dict(tensor=dict(scale=float("nan")))], ids=str)
def test_muon_refuses(kw):
    refused(muon(**kw))


def test_muon_limits_workspace_and_nothing():
    refused(muon(tensor=dict(rows=65537)), "EMB_ERR_UNSUPPORTED")
    refused(muon(ws=None), "EMB_ERR_WORKSPACE")
    refused(muon(wsb=100), "EMB_ERR_WORKSPACE")
    refused(muon(ws=P + 128), "EMB_ERR_WORKSPACE")
    refused(E.lib().emb_muon_step(None, None, 0, None, None, 0, None))
    assert muon(n=0) == 0
    assert muon(tensor=dict(rows=0, p=None, m=None), grads=None, ws=None, wsb=0) == 0
    with pytest.raises(ValueError):
        E.Muon([])
    with pytest.raises(ValueError):
        E.Muon([torch.zeros(3)])
    with pytest.raises(ValueError):
        E.Muon([torch.zeros(3, 4)])             # host memory
    with pytest.raises(KeyError):
        E.Muon([torch.zeros(3, 4)], products="double")


def tok_fwd(**kw):
    a = dict(w=P, wt=0, v=10, d=8, ldw=8, t=P, tt=0, n=5, pad=-1, s=1.0, out=P, ot=0, ldo=8)
    a.update(kw)
    return E.lib().emb_token_fwd(*[a[k] for k in ("w", "wt", "v", "d", "ldw", "t", "tt", "n", "pad", "s", "out", "ot", "ldo")], None)


def tok_bwd(**kw):
    a = dict(g=P, gt=0, ldg=8, t=P, tt=0, n=5, pad=-1, v=10, d=8, s=1.0, acc=0, dw=P, wt=0, ldw=8, ws=P, wsb=1 << 40)
    a.update(kw)
    return E.lib().emb_token_bwd(*[a[k] for k in ("g", "gt", "ldg", "t", "tt", "n", "pad", "v", "d", "s", "acc", "dw", "wt", "ldw", "ws", "wsb")], None)


COMMON = [dict(wt=3), dict(tt=2), dict(n=-1), dict(v=-1), dict(d=-1), dict(t=None), dict(t=P + 2), dict(tt=1, t=P + 4), dict(ldw=7)]


@pytest.mark.parametrize("kw", COMMON + [dict(ot=-1), dict(w=None), dict(out=None), dict(w=P + 2), dict(out=P + 1), dict(ldo=7)], ids=str)
def test_token_fwd_refuses(kw):
    refused(tok_fwd(**kw))


@pytest.mark.parametrize("kw", COMMON + [dict(gt=4), dict(g=None), dict(dw=None), dict(g=P + 2), dict(dw=P + 2), dict(ldg=7)], ids=str)
def test_token_bwd_refuses(kw):
    refused(tok_bwd(**kw))


def test_token_limits_workspace_and_nothing():
    for kw in (dict(n=1 << 30), dict(v=1 << 31), dict(d=65537, ldw=65537, ldo=65537)):
        refused(tok_fwd(**kw), "EMB_ERR_UNSUPPORTED")
    for kw in (dict(n=1 << 30), dict(v=1 << 31), dict(d=65537, ldw=65537, ldg=65537)):
        refused(tok_bwd(**kw), "EMB_ERR_UNSUPPORTED")
    for kw in (dict(ws=None), dict(wsb=64), dict(ws=P + 16)):
        refused(tok_bwd(**kw), "EMB_ERR_WORKSPACE")
    refused(E.lib().emb_token_bwd_workspace_size(1, 1, 1, None))
    assert tok_fwd(n=0) == 0 and tok_fwd(d=0, ldw=0, ldo=0) == 0
    assert tok_bwd(v=0) == 0 and tok_bwd(n=0, acc=1, g=None, t=None, ws=None, wsb=0) == 0
    assert E.emb_token_bwd_workspace_size(0, 5, 5) == 0 and E.emb_token_bwd_workspace_size(1000, 5, 8) > 0


def test_binding_checks_shapes_and_types():
    z = torch.zeros
    with pytest.raises(ValueError):
        E.emb_fp4_quantize(z(4, 4))
    with pytest.raises(ValueError):
        E.emb_token_fwd(z(4, 4), z(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        E.emb_token_bwd(z(3, 4), z(3, dtype=torch.int64), 4)


def calls(where):
    """Each operator with its tensors on the GPUs that `where` names (default 0)."""
    w = lambda k, t: on(where.get(k, 0), t)  # noqa: E731
    z = torch.zeros
    u8, i64 = torch.uint8, torch.int64
    sc = lambda r, c: z(-(-r // 128), -(-c // 128), 32, 4, 4, dtype=u8)  # noqa: E731
    return {
        "quantize": lambda: E.emb_fp4_quantize(w("x", z(4, 6))),
        "dequantize": lambda: E.emb_fp4_dequantize(w("q", z(4, 16, dtype=u8)), w("s", sc(4, 32)), out=w("out", z(4, 32))),
        "matmul": lambda: E.emb_fp4_matmul(w("a", z(4, 16, dtype=u8)), w("sa", sc(4, 32)), w("b", z(8, 16, dtype=u8)), w("sb", sc(8, 32)),
                                           bias=w("bias", z(8)), out=w("out", z(4, 8)), workspace=w("workspace", z(64))),
        "fwd": lambda: E.emb_token_fwd(w("weight", z(9, 6)), w("tokens", z(4, dtype=i64)), out=w("out", z(4, 6))),
        "bwd": lambda: E.emb_token_bwd(w("grad", z(4, 6)), w("tokens", z(4, dtype=i64)), 9, out=w("out", z(9, 6)), workspace=w("workspace", z(4000))),
    }


@pytest.mark.parametrize("op,names", [("quantize", "x"), ("dequantize", "q s out"), ("matmul", "a sa b sb bias out workspace"),
                                      ("fwd", "weight tokens out"), ("bwd", "grad tokens out workspace")])
def test_operands_on_another_device_are_refused(monkeypatch, op, names):
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


def test_constants_match_the_header():
    text = open(E.HEADER).read()
    for name in ("EMB_FP4_BLOCK", "EMB_MUON_MAX_DIM", "EMB_MAX_TOKENS", "EMB_FLAG_BAD_TOKEN"):
        assert int(re.search(rf"^#define {name}\s+(\d+)", text, re.M).group(1)) == getattr(E, name)


class Reads:
    """The library as far as a launch, which reads rows of codes as the kernels do: in whole 16 bytes."""

    def __init__(self, lib, short):
        self.lib, self.short, self.rows = lib, {t.data_ptr() for t in short}, []

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return getattr(self.lib, name)

        def launched(*args):
            k = {"emb_fp4_dequantize": lambda q, ld, s, r, c, *_: [(q, ld, r, -(-c // 2))],
                 "emb_fp4_matmul": lambda a, lda, sa, b, ldb, sb, m, n, k, *_: [(a, lda, m, -(-k // 2)), (b, ldb, n, -(-k // 2))]}[name](*args)
            for at, ld, rows, width in k:
                assert at not in self.short, "reads past the end of a tensor"
                assert ld % 16 == 0
                whole = -(-width // 16) * 16
                self.rows.append([ctypes.string_at(at + i * ld, whole)[:width] for i in range(rows)])
            return 0
        return launched


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("width", [1, 15, 20, 500])
def test_rows_are_not_read_past_their_storage(monkeypatch, rows, width):
    """Codes whose storage ends with the last row's last byte are laid out anew; others are taken as they are."""
    ld = -(-width // 16) * 16
    g = torch.Generator().manual_seed(width)
    short = torch.randint(0, 256, ((rows - 1) * ld + width,), dtype=torch.uint8, generator=g).as_strided((rows, width), (ld, 1))
    room = torch.randint(0, 256, (5, ld), dtype=torch.uint8, generator=g)[:, :width]
    sc = lambda r: torch.zeros(1, -(-2 * width // 128), 32, 4, 4, dtype=torch.uint8)  # noqa: E731
    stub = Reads(E.lib(), [short])
    monkeypatch.setattr(E, "lib", lambda: stub)
    monkeypatch.setattr(E, "_current_device", lambda: 0)
    monkeypatch.setattr(E, "_raw_stream", lambda stream, dev=None: 0)
    want = [bytes(r.tolist()) for r in short]
    assert E.emb_fp4_dequantize(on(0, short), on(0, sc(rows)), out=on(0, torch.zeros(rows, 2 * width))).shape == (rows, 2 * width)
    for a, b in ((short, room), (room, short)):
        E.emb_fp4_matmul(on(0, a), on(0, sc(1)), on(0, b), on(0, sc(1)), out=on(0, torch.zeros(a.shape[0], b.shape[0])))
    assert stub.rows[0] == want and stub.rows[1] == want and stub.rows[4] == want
    assert stub.rows[2] == stub.rows[3] == [bytes(r.tolist()) for r in room]
    kept = torch.zeros(1, ld, dtype=torch.uint8)[:, :width]
    assert E._packed(on(0, kept), "q", 0, None)[0].data_ptr() == kept.data_ptr()      # there is room: no copy


def test_rows_that_the_library_refuses_are_left_to_it():
    """Off the alignment, over one another or at odd distances: refused where the storage ends with them as elsewhere."""
    for off, rows, ld in ((1, 1, 32), (8, 3, 32), (0, 3, 0), (0, 3, 16), (0, 3, 20)):
        for end in (off + (rows - 1) * ld + 20, 400):      # with the last row's last byte, or later
            hold = torch.zeros(end, dtype=torch.uint8)
            assert hold.data_ptr() % 16 == 0
            t = hold.as_strided((rows, 20), (ld, 1), off)
            got, dist = E._packed(on(0, t), "q", 0, None)
            assert got.data_ptr() == t.data_ptr()
            refused(back(q=got.data_ptr(), ldq=dist, rows=rows, cols=40, out=P, ldo=40))
