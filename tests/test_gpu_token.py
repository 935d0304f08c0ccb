"""Rows by token with a scale, and the matrix's gradient, against 64 bits."""
import pytest
import torch

import sparse_ctr_embedding_gb300 as E

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    E.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def ids(n, vocab, seed, kind=torch.int64, pad=0.2, hot=0.0):
    g = torch.Generator().manual_seed(seed)
    t = (float(vocab) ** torch.rand(n, generator=g, dtype=torch.float64) - 1).long().clamp(0, vocab - 1)
    t = (t * 7919 + 3) % vocab
    t[torch.rand(n, generator=g) < hot] = vocab // 2
    t[torch.rand(n, generator=g) < pad] = -1
    return t.to(kind).cuda()


def grad64(grad, tokens, vocab, scale):
    """The gradient, and the sum of the magnitudes that make it up."""
    t, g = tokens.reshape(-1).long(), grad.reshape(tokens.numel(), -1).double()
    keep = t >= 0
    out = torch.zeros(vocab, g.shape[1], dtype=torch.float64, device="cuda")
    return (out.index_put((t[keep],), g[keep], accumulate=True) * scale, out.index_put((t[keep],), g[keep].abs(), accumulate=True) * abs(scale))


def held(got, ref, size, tokens, vocab):
    """A sum of c values takes c - 1 additions, joined pieces included, and the scale one
    rounding; the result one to its own type."""
    t = tokens.reshape(-1).long()
    count = torch.bincount(t[t >= 0], minlength=vocab).double()[:, None]
    tol = (count + 2) * U * size + torch.finfo(got.dtype).eps / 2 * ref.abs() * (got.dtype != F32) + 2.0 ** -25 * (got.dtype == F16)
    assert bool(((got.double() - ref).abs() <= tol).all())
    assert bool((got[(count == 0)[:, 0]] == 0).all())


@pytest.mark.parametrize("dim", [1, 3, 4, 8, 12, 64, 100, 128, 257, 1024, 2056])
@pytest.mark.parametrize("weight,out", [(F32, F32), (F32, BF16), (BF16, F16), (F16, BF16)])
def test_lookup(dim, weight, out):
    vocab = 300
    w = torch.randn(vocab, dim, generator=torch.Generator().manual_seed(dim)).to(weight).cuda()
    for kind in (torch.int32, torch.int64):
        for shape in ((1,), (50,), (7, 33), (0,)):
            n = torch.Size(shape).numel()
            t = ids(n, vocab, dim + n, kind).view(shape)
            got = E.emb_token_fwd(w, t, scale=1.7, out_dtype=out)
            assert got.shape == (*shape, dim) and got.dtype == out
            scale = torch.tensor(1.7, device="cuda")
            want = torch.where((t >= 0)[..., None], w[t.clamp_min(0).long()].float() * scale, 0.0).to(out)   # one product, one rounding
            assert torch.equal(got, want)
    assert E.emb_check_op_flag() == 0


SIZES = [(1, 1, 4), (1, 1000, 16), (50, 7, 64), (63, 5, 8), (64, 1, 8), (65, 1, 8), (1000, 300, 1), (1000, 300, 3), (4096, 200, 100), (4097, 65536, 4),
         (5000, 65537, 12), (30000, 1 << 20, 32), (30000, 201, 128), (2000, 40, 1000), (2000, 40, 2056), (100000, 3, 5), (70000, 1 << 24, 1)]


@pytest.mark.parametrize("n,vocab,dim", SIZES)
@pytest.mark.parametrize("grad,weight", [(F32, F32), (BF16, F32), (F16, BF16), (BF16, F16)])
def test_gradient(n, vocab, dim, grad, weight):
    for kind, pad, hot in ((torch.int64, 0.2, 0.0), (torch.int32, 0.0, 0.7)):
        t = ids(n, vocab, n + dim, kind, pad, hot)
        g = torch.randn(n, dim, generator=torch.Generator().manual_seed(n)).to(grad).cuda()
        got = E.emb_token_bwd(g, t, vocab, scale=0.37, dtype=weight)
        held(got, *grad64(g, t, vocab, 0.37), t, vocab)
        assert torch.equal(got, E.emb_token_bwd(g, t, vocab, scale=0.37, dtype=weight))
    assert E.emb_check_op_flag() == 0


def test_gradient_of_many_tokens():
    n, vocab, dim = 1_000_003, 500_000, 16
    t = ids(n, vocab, 1, pad=0.3, hot=0.1)
    g = torch.randn(n, dim, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    ws = torch.full((E.emb_token_bwd_workspace_size(n, vocab, dim),), 0xA5, dtype=torch.uint8, device="cuda")
    a = E.emb_token_bwd(g, t, vocab, workspace=ws)
    held(a, *grad64(g, t, vocab, 1.0), t, vocab)
    for _ in range(3):
        assert torch.equal(a, E.emb_token_bwd(g, t, vocab, workspace=ws))


def test_only_padding_and_no_tokens():
    for n in (0, 5, 5000):
        t = torch.full((n,), -1, device="cuda")
        out = torch.full((40, 12), 3.0, device="cuda")
        g = torch.randn(n, 12, device="cuda")
        E.emb_token_bwd(g, t, 40, out=out, accumulate=True)
        assert bool((out == 3.0).all())
        E.emb_token_bwd(g, t, 40, out=out)
        assert bool((out == 0).all())
    assert E.emb_token_fwd(torch.zeros(0, 8, device="cuda"), torch.full((3,), -1, device="cuda")).tolist() == [[0.0] * 8] * 3
    assert E.emb_check_op_flag() == 0


def test_padding_row_and_bad_tokens():
    w = torch.randn(10, 8, device="cuda")
    t = torch.tensor([0, 3, 9, 3, 5], device="cuda")
    out = E.emb_token_fwd(w, t, padding=3)
    assert bool((out[[1, 3]] == 0).all()) and torch.equal(out[[0, 2, 4]], w[[0, 9, 5]])
    g = torch.randn(5, 8, device="cuda")
    dw = E.emb_token_bwd(g, t, 10, padding=3)
    assert bool((dw[3] == 0).all()) and torch.equal(dw[[0, 9, 5]], g[[0, 2, 4]])
    assert E.emb_check_op_flag() == 0
    for bad in (10, -2, 1 << 40, -(1 << 62)):
        t[1] = bad
        out = E.emb_token_fwd(w, t)
        assert bool((out[1] == 0).all()) and torch.equal(out[[0, 2, 3, 4]], w[[0, 9, 3, 5]])
        assert E.emb_check_op_flag() == E.EMB_FLAG_BAD_TOKEN and E.emb_check_op_flag() == 0
        dw = E.emb_token_bwd(g, t, 10)
        assert torch.equal(dw[3], g[3]) and torch.equal(dw[9], g[2]) and bool((dw[1] == 0).all())
        assert E.emb_check_op_flag() == E.EMB_FLAG_BAD_TOKEN and E.emb_check_op_flag() == 0


@pytest.mark.parametrize("weight", [F32, BF16])
def test_accumulate_strides_and_unaligned(weight):
    n, vocab, dim = 3000, 90, 24
    t = ids(n, vocab, 4)
    g = torch.randn(n, 2 * dim + 1, device="cuda")[:, 1:1 + dim]
    hold = torch.full((vocab, dim + 9), 2.0, dtype=weight, device="cuda")
    for view in (hold[:, 8:8 + dim], hold[:, 1:1 + dim]):
        hold.fill_(2.0)
        ref, size = grad64(g, t, vocab, 1.0)
        E.emb_token_bwd(g, t, vocab, out=view, accumulate=True)
        count = torch.bincount(t[t >= 0], minlength=vocab).double()[:, None]
        tol = (count + 3) * U * (size + 2) + (torch.finfo(weight).eps / 2 * (ref + 2).abs() if weight != F32 else 0)
        assert bool(((view.double() - ref - 2).abs() <= tol).all())
        E.emb_token_bwd(g, t, vocab, out=view)
        held(view, ref, size, t, vocab)
        view.fill_(2.0)
        assert bool((hold == 2.0).all())
        w = torch.randn(vocab, dim + 9, device="cuda").to(weight)[:, 1:1 + dim]
        out = torch.full((n, dim + 3), 5.0, device="cuda")
        E.emb_token_fwd(w, t, out=out[:, :dim])
        assert torch.equal(out[:, :dim], torch.where((t >= 0)[:, None], w[t.clamp_min(0)].float(), 0.0)) and bool((out[:, dim:] == 5.0).all())


def test_graph_stream_and_differences():
    """Captured and on another stream; the gradient is the loss's derivative, by its differences
    (the loss <g, scale W[t]> is linear in W: differences are exact up to rounding)."""
    n, vocab, dim = 700, 50, 20
    t = ids(n, vocab, 5)
    g, w = torch.randn(n, dim, device="cuda"), torch.randn(vocab, dim, device="cuda")
    want, out = E.emb_token_bwd(g, t, vocab, scale=3.0), E.emb_token_fwd(w, t, scale=3.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b = E.emb_token_bwd(g, t, vocab, scale=3.0, stream=s), E.emb_token_fwd(w, t, scale=3.0, stream=s)
    s.synchronize()
    assert torch.equal(a, want) and torch.equal(b, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = E.emb_token_bwd(g, t, vocab, scale=3.0)
        b = E.emb_token_fwd(w, t, scale=3.0)
    t.copy_(t.flip(0).clone())
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, E.emb_token_bwd(g, t, vocab, scale=3.0)) and torch.equal(b, E.emb_token_fwd(w, t, scale=3.0))
    loss = lambda w: float((g.double() * E.emb_token_fwd(w, t, scale=3.0).double()).sum())  # noqa: E731
    for v, c in ((int(t[0].clamp_min(0)), 0), (7, 19), (49, 3)):
        up, down = w.clone(), w.clone()
        up[v, c], down[v, c] = 1.0, -1.0
        slope = (loss(up) - loss(down)) / 2
        size = float((g.double().abs() * (t == v)[:, None])[:, c].sum()) * 3
        assert abs(slope - float(a[v, c])) <= 1e-4 * (size + 1)


@pytest.mark.parametrize("dim", [5, 64])
@pytest.mark.parametrize("accumulate", [False, True])
def test_a_wait_that_runs_out(dim, accumulate):
    """The flag is raised and no row is summed: the gradient is zeros, or stays what it was."""
    n, vocab = 20000, 70000            # five tiles of the sort, three passes
    t = ids(n, vocab, dim, hot=0.3)
    g = torch.randn(n, dim, generator=torch.Generator().manual_seed(dim)).cuda()
    want = E.emb_token_bwd(g, t, vocab)
    for tile in (1, 4):
        out = torch.full((vocab, dim), 0.25, device="cuda")
        try:
            E.emb_debug_lose_op_wait("load", tile)
            E.emb_token_bwd(g, t, vocab, out=out, accumulate=accumulate)
        finally:
            E.emb_debug_lose_op_wait(None)
        assert E.emb_check_op_flag() == E.EMB_FLAG_OP_TIMEOUT
        assert bool((out == (0.25 if accumulate else 0.0)).all())
        assert torch.equal(E.emb_token_bwd(g, t, vocab), want)
        assert E.emb_check_op_flag() == 0


@pytest.mark.parametrize("dim", [5, 12, 64])
@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
@pytest.mark.parametrize("vocab", [201, 70_001])
def test_bad_tokens_among_many(dim, kind, vocab):
    """Tokens that name no row, in every tile of the sort and between equal tokens: counted nowhere, summed
    nowhere, whatever row their low bits would name; the others' sums are those without them."""
    n = 20_001
    t = ids(n, vocab, dim, kind, pad=0.1, hot=0.3)
    low, high = (-(1 << 31), (1 << 31) - 1) if kind == torch.int32 else (-(1 << 62), 1 << 62)
    bad = [vocab, vocab + 1, vocab + 256, 65_536 * 4, -2, -256, low, high, high - 255] + ([1 << 32, (1 << 40) + 7, -(1 << 32)] if kind == torch.int64 else [])
    at = torch.randperm(n, generator=torch.Generator().manual_seed(vocab))[:5000].cuda()
    at = torch.cat([at, torch.tensor([0, 4095, 4096, n - 1], device="cuda")])
    t[at] = torch.tensor(bad, device="cuda").to(kind)[torch.arange(len(at), device="cuda") % len(bad)]
    clean = torch.where((t >= 0) & (t < vocab), t, -1)
    assert int((clean >= 0).sum()) > 5000
    g = torch.randn(n, dim, generator=torch.Generator().manual_seed(dim)).cuda()
    g[clean < 0] = float("nan")                    # their gradients are not read
    for padding in (-1, vocab // 2):               # the second one: the token that occurs most
        keep = torch.where(clean == padding, -1, clean)
        ref, size = grad64(g, keep, vocab, 0.5)
        got = E.emb_token_bwd(g, t, vocab, scale=0.5, padding=padding)
        assert E.emb_check_op_flag() == E.EMB_FLAG_BAD_TOKEN and E.emb_check_op_flag() == 0
        held(got, ref, size, keep, vocab)
        assert torch.equal(got, E.emb_token_bwd(g, keep, vocab, scale=0.5)) and E.emb_check_op_flag() == 0
        out = torch.full((vocab, dim), 2.0, device="cuda")
        E.emb_token_bwd(g, t, vocab, scale=0.5, padding=padding, out=out, accumulate=True)
        seen = torch.zeros(vocab, dtype=torch.bool, device="cuda")
        seen[keep[keep >= 0].long()] = True
        assert bool((out[~seen] == 2.0).all()) and torch.equal(out[seen], got[seen] + 2.0)
        w = torch.randn(vocab, dim, device="cuda")
        rows = E.emb_token_fwd(w, t, padding=padding)
        assert torch.equal(rows, torch.where((keep >= 0)[:, None], w[keep.clamp_min(0).long()], 0.0))
        assert E.emb_check_op_flag() == E.EMB_FLAG_BAD_TOKEN
    t.fill_(vocab)
    assert bool((E.emb_token_bwd(g, t, vocab) == 0).all()) and E.emb_check_op_flag() == E.EMB_FLAG_BAD_TOKEN
