"""The dense operators and the embedding step together, as examples/dense_tower.py runs them."""
import importlib.util
import os

import pytest
import torch

import sparse_ctr_embedding_gb300 as E

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tower():
    E.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "dense_tower.py")
    spec = importlib.util.spec_from_file_location("dense_tower", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("state", ["f32", "q8"])
def test_training_fits_its_batch(tower, state):
    losses = tower.train(steps=60, state=state)
    # an untrained logit of 0 costs ln 2; labels are drawn with probability 0.3 (entropy 0.61), so only a
    # model that tells the samples apart gets well below that
    assert abs(losses[0] - 0.6931) < 1e-3
    assert losses[-1] < 0.3 and losses[-1] < min(losses[:10])
    assert tower.train(steps=3, state=state) == losses[:3]      # a step repeats bitwise


def test_gradients_of_the_tower_against_autograd(tower):
    """The 8-bit tower's gradients against float64 autograd of the same network:
    each product's operands carry up to 2^-4 of rounding, independent from
    element to element, so every gradient as a whole stays within a tenth."""
    g = torch.Generator(device="cuda").manual_seed(3)
    t = tower.Tower(192, 256, 2, seed=3, state="f32")
    t.p["w_out"].copy_(torch.randn(256, device="cuda", generator=g) / 16)
    pooled = torch.randn(384, 192, device="cuda", generator=g)
    dlogits = torch.randn(384, device="cuda", generator=g) / 384
    q = {k: v.double().requires_grad_() for k, v in t.p.items()}
    x0 = pooled.double().requires_grad_()
    rms = lambda z: z * (z.square().mean(1, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
    x = x0 @ q["w_in"].t() + q["b_in"]
    h = rms(x) * q["pre0"]
    for i in range(2):
        x = x + torch.sigmoid(h @ q[f"w_g{i}"].t()) * rms(h @ q[f"w_f{i}"].t()) * q[f"post{i}"]
        h = rms(x) * q[f"pre{i + 1}"]
    want = h @ q["w_out"]
    got = t.forward(pooled)
    assert float((got.double() - want).norm() / want.norm()) < 0.1
    seen = {}
    t.opt.step = lambda grads: seen.update(zip(t.names, grads))
    dpooled = t.backward(dlogits)
    ref = dict(zip(["pooled"] + t.names, torch.autograd.grad(want, [x0] + [q[n] for n in t.names], dlogits.double())))
    seen["pooled"] = dpooled
    for n, r in ref.items():
        assert float((seen[n].double() - r).norm() / r.norm()) < 0.1, n
