"""4-bit codes and plain embeddings past 2^31 and 2^32 elements, and calls that overlap on the GPU."""
import pytest
import torch

import sparse_ctr_embedding_gb300 as E
from fp4_ref import encode, unpack, untile, values

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    E.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def test_codes_past_2_32_elements():
    rows, cols = 70_001, 65_536           # 4.6e9 elements, 2.3e9 bytes of codes
    x = torch.empty(rows, cols, dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for r in range(0, rows, 10_000):
        x[r:r + 10_000] = torch.randn(min(10_000, rows - r), cols, device="cuda", generator=g)
    q, s, qt, st = E.emb_fp4_quantize(x, transpose=True)
    back, back_t = E.emb_fp4_dequantize(q, s), E.emb_fp4_dequantize(qt, st, rows)
    for r in (0, 1, 127, 32_768, 65_535, 65_536, 69_999, 70_000):
        code, byte = encode(x[r:r + 1].cpu(), 1)
        assert torch.equal(back[r].cpu().double(), values(code, byte)[0])
        assert torch.equal(unpack(q[r:r + 1], cols), code)
    for c in (0, 5, 32_767, 65_535):
        code, byte = encode(x[:, c].cpu()[None], 1)
        assert torch.equal(back_t[c].cpu().double(), values(code, byte)[0])
    del back, back_t, x
    # products that start past 2^31 bytes of codes
    w, sw = E.emb_fp4_quantize(torch.randn(96, cols, device="cuda", generator=g))
    out = E.emb_fp4_matmul(q, s, w, sw, out_dtype=F32)
    B = values(unpack(w, cols), untile(sw, 96, cols // 32)).cuda()
    for r in (0, 69_888, 70_000):
        A = values(unpack(q[r:r + 1], cols), untile(s[r // 128:r // 128 + 1], r % 128 + 1, cols // 32)[r % 128:]).cuda()
        ref, size = (A @ B.t())[0], (A.abs() @ B.abs().t())[0]
        assert bool(((out[r].double() - ref).abs() <= (128 + 2 * cols // 64 + 320) * 2.0 ** -24 * size).all())


def test_rows_past_2_32_elements():
    vocab, dim = 70_000_000, 64           # 4.5e9 elements
    w = torch.zeros(vocab, dim, dtype=BF16, device="cuda")
    at = torch.tensor([0, 1, 33_554_431, 33_554_432, 67_108_863, 67_108_864, 69_999_999, 69_999_999, 5], device="cuda")
    w[at] = torch.randn(len(at), dim, device="cuda").to(BF16)
    assert torch.equal(E.emb_token_fwd(w, at), w[at])
    g = torch.randn(len(at), dim, device="cuda")
    w.fill_(1.0)
    E.emb_token_bwd(g, at, vocab, out=w)
    want = g.clone()
    want[6] = want[7] = g[6] + g[7]
    assert torch.equal(w[at], want.to(BF16))
    w[at] = 0
    assert not bool(w.any())


def test_gradients_past_2_31_elements():
    n, vocab, dim = 17_000_000, 1000, 128          # 2.2e9 elements of gradients
    g = torch.Generator(device="cuda").manual_seed(2)
    t = torch.randint(0, vocab, (n,), device="cuda", generator=g, dtype=torch.int32)
    grad = torch.randn(n, 1, device="cuda", generator=g).to(BF16).expand(n, dim).contiguous()
    dw = E.emb_token_bwd(grad, t, vocab)
    want = torch.zeros(vocab, dtype=torch.float64, device="cuda").index_put((t.long(),), grad[:, 0].double(), accumulate=True)
    size = torch.zeros(vocab, dtype=torch.float64, device="cuda").index_put((t.long(),), grad[:, 0].double().abs(), accumulate=True)
    # chunks of 64 additions, then their sums one after the other in up to 16 shares: c / 64 at most
    count = torch.bincount(t, minlength=vocab).double()
    assert bool(((dw.double() - want[:, None]).abs() <= ((64 + count / 64 + 32) * 2.0 ** -24 * size)[:, None]).all())
    assert torch.equal(dw, E.emb_token_bwd(grad, t, vocab))


def test_calls_that_overlap():
    """The same operators on two streams at a time, each with buffers of its own: cooperative launches,
    pairs of SMs, tiles that wait for tiles before them."""
    shapes = [(300, 700), (512, 512), (64, 100)]
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    grads = [[rand(*s) for s in shapes] for _ in range(2)]
    x, w = rand(5000, 2048), rand(600, 2048)
    (a, sa), (b, sb) = E.emb_fp4_quantize(x), E.emb_fp4_quantize(w)
    t = torch.randint(0, 3000, (100_000,), device="cuda", generator=g)
    tg = rand(100_000, 32)

    def work(opt, i, stream):
        opt.step(grads[i], stream=stream)
        y = E.emb_fp4_matmul(a, sa, b, sb, stream=stream)
        dw = E.emb_token_bwd(tg, t, 3000, stream=stream)
        opt.step(grads[i], stream=stream)
        return y, dw

    def fresh():
        return [E.Muon([torch.ones(s, device="cuda") for s in shapes], lr=0.1) for _ in range(2)]

    want_opts = fresh()
    want = [work(o, i, None) for i, o in enumerate(want_opts)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        opts = fresh()
        torch.cuda.synchronize()
        got = [work(o, i, streams[i]) for i, o in enumerate(opts)]
        torch.cuda.synchronize()
        assert E.emb_check_op_flag() == 0
        for i in range(2):
            assert all(torch.equal(p, q) for p, q in zip(got[i], want[i]))
            assert all(torch.equal(p, q) for p, q in zip(opts[i].params, want_opts[i].params))
