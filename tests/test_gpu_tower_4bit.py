"""The 4-bit layer, the plain embeddings and both optimizers as one step runs them."""
import importlib.util
import os

import pytest
import torch

import sparse_ctr_embedding_gb300 as E
from fp4_ref import ulps, unpack, untile, values
from muon_ref import momentum, orthogonal

pytestmark = pytest.mark.gpu
F32 = torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    E.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def matrix(q, s):
    cols = 2 * q.shape[1]
    return values(unpack(q, cols), untile(s, q.shape[0], -(-cols // 32))).cuda()


def near(got, ref, size, n):
    assert bool(((got.double() - ref).abs() <= n * U * size + 1e-30).all())


def test_a_step_of_one_layer():
    """tokens -> rows -> 4-bit layer -> gradients -> Muon for its matrix, AdamW for the embedding; the
    second step works on what the first one left.  Each stage against 64 bits of what it was given."""
    B, V, D, O = 384, 70, 160, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    emb, w = rand(V, D) * 0.1, rand(O, D) * D ** -0.5
    muon, adamw = E.Muon([w], lr=0.01, weight_decay=0.1, products="split"), E.AdamW([emb], lr=0.01, weight_decay=0.0)
    m = torch.zeros(O, D, dtype=torch.float64, device="cuda")
    for step in range(2):
        tokens = torch.randint(-1, V, (B,), device="cuda", generator=g)
        dy = rand(B, O) * 0.01
        x = E.emb_token_fwd(emb, tokens, scale=D ** 0.5)
        qx, sx, qxt, sxt = E.emb_fp4_quantize(x, 1, transpose=True)
        qw, sw, qwt, swt = E.emb_fp4_quantize(w, 32, transpose=True)
        qd, sd, qdt, sdt = E.emb_fp4_quantize(dy, 1, transpose=True)
        y = E.emb_fp4_matmul(qx, sx, qw, sw, out_dtype=F32)
        dx = E.emb_fp4_matmul(qd, sd, qwt, swt, out_dtype=F32)
        dw = E.emb_fp4_matmul(qdt, sdt, qxt, sxt, out_dtype=F32)
        demb = E.emb_token_bwd(dx, tokens, V, scale=D ** 0.5)
        before, emb0 = w.double(), emb.clone()
        muon.step([dw])
        adamw.step([demb])
        X, W, G = matrix(qx, sx), matrix(qw, sw), matrix(qd, sd)
        assert torch.equal(matrix(qwt, swt).t(), W)
        near(y, X @ W.t(), X.abs() @ W.abs().t(), ulps(D))
        near(dx, G @ W, G.abs() @ W.abs(), ulps(O))
        Gt, Xt = matrix(qdt, sdt), matrix(qxt, sxt)
        near(dw, Gt @ Xt.t(), Gt.abs() @ Xt.abs().t(), ulps(B))
        keep = tokens >= 0
        ref = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_put((tokens[keep],), dx[keep].double(), accumulate=True) * D ** 0.5
        size = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_put((tokens[keep],), dx[keep].double().abs(), accumulate=True) * D ** 0.5
        near(demb, ref, size, B + 2)
        m, u = momentum(dw, m, 0.95)
        want = before * (1 - 0.01 * 0.1) - 0.01 * 0.2 * max(O, D) ** 0.5 * orthogonal(u)
        # the update's own error is that of float32 products: 1e-4 of its largest entry (test_gpu_muon)
        assert float((w.double() - want).abs().max()) <= 1e-4 * 0.01 * 0.2 * max(O, D) ** 0.5 + 4 * U * float(before.abs().max())
        assert not torch.equal(emb, emb0)
        absent = torch.ones(V, dtype=torch.bool, device="cuda")
        absent[tokens[keep]] = False
        if step == 0:
            assert torch.equal(emb[absent], emb0[absent])      # no gradient yet: AdamW leaves them
    assert E.emb_check_op_flag() == 0


@pytest.fixture(scope="module")
def tower():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "dense_tower.py")
    spec = importlib.util.spec_from_file_location("dense_tower4", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("layers,matrices,positions", [("fp4", "muon", 7), ("fp4", "adamw", 0), ("fp8", "muon", 3)])
def test_the_example_runs(tower, layers, matrices, positions):
    losses = tower.train(steps=4, layers=layers, matrices=matrices, positions=positions)
    assert len(losses) == 4 and all(0.0 < v < 10.0 for v in losses)
    assert tower.train(steps=2, layers=layers, matrices=matrices, positions=positions) == losses[:2]      # a step repeats bitwise


def test_gradients_of_the_example(tower):
    """The 4-bit tower's gradients against float64 autograd of the same network.  An operand's rounding is at
    most a quarter of its value (half a step of 0.5 at 1), evenly spread about an eighth as a root mean square,
    independent from element to element; a gradient has come through up to six such products, both operands
    rounded: sqrt(12) / 8 = 0.43 of its norm."""
    g = torch.Generator(device="cuda").manual_seed(3)
    t = tower.Tower(192, 256, 2, seed=3, state="f32", layers="fp4", positions=5)
    t.p["w_out"].copy_(torch.randn(256, device="cuda", generator=g) / 16)
    pooled = torch.randn(384, 192, device="cuda", generator=g)
    dlogits = torch.randn(384, device="cuda", generator=g) / 384
    at = torch.randint(0, 5, (384,), device="cuda", generator=g)
    q = {k: v.double().requires_grad_() for k, v in t.p.items()}
    x0 = pooled.double().requires_grad_()
    rms = lambda z: z * (z.square().mean(1, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
    x = x0 @ q["w_in"].t() + q["b_in"] + q["pos"][at] * 16
    h = rms(x) * q["pre0"]
    for i in range(2):
        x = x + torch.sigmoid(h @ q[f"w_g{i}"].t()) * rms(h @ q[f"w_f{i}"].t()) * q[f"post{i}"]
        h = rms(x) * q[f"pre{i + 1}"]
    want = h @ q["w_out"]
    t.forward(pooled, at)
    seen = {}
    t.step = seen.update
    seen["pooled"] = t.backward(dlogits)
    ref = dict(zip(["pooled"] + t.names, torch.autograd.grad(want, [x0] + [q[n] for n in t.names], dlogits.double())))
    for n, r in ref.items():
        assert float((seen[n].double() - r).norm() / r.norm()) < 0.43, n
