"""The 8-bit quantiser (bit for bit) and matrix product (against 64 bits)."""
import pytest
import torch

import sparse_ctr_embedding_gb300 as E
from dense_ref import U, block_scales, close, dequant64

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    E.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def bits(t):
    return t.cpu().contiguous().view(torch.uint8)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (2, 129), (127, 64), (128, 128), (129, 257), (300, 1000), (5, 4099),
                                       (1030, 16)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize(rows, cols, dtype, block_rows):
    g = torch.Generator().manual_seed(rows * cols)
    x = (torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))).to(dtype)
    x[0, 0] = 0.0
    q, s, qt, st = E.emb_fp8_quantize(x.cuda(), block_rows=block_rows, transpose=True)
    for got, scale, src in ((q, s, x), (qt, st, x.t())):
        rq, rs = block_scales(src, block_rows)
        assert torch.equal(scale.cpu(), rs)
        assert torch.equal(bits(got), bits(rq))
        pad = torch.as_strided(got.view(torch.uint8), (got.shape[0], got.stride(0)), (got.stride(0), 1))[:, got.shape[1]:]
        assert bool((pad == 0).all())       # up to the row's next 16 bytes
        # the values that the codes stand for are within half a step of x
        err = (dequant64(got.cpu(), scale.cpu()) - src.double()).abs()
        full = dequant64(torch.ones_like(rq.float()).to(rq.dtype), rs)     # one code unit
        assert bool((err <= src.double().abs() * 2.0 ** -4 * (1 + 1e-6) + full * 2.0 ** -10 * (1 + 1e-6) + 1e-37).all())
    q1, s1 = E.emb_fp8_quantize(x.cuda(), block_rows=block_rows)
    assert torch.equal(bits(q1), bits(q)) and torch.equal(s1, s)


def test_quantize_special_values():
    x = torch.randn(256, 256, generator=torch.Generator().manual_seed(1))
    x[0, :128] = 0.0
    x[1, 5], x[1, 130] = float("inf"), float("nan")
    x[2, :128] = 1e-42
    x[3, 3] = 3e38
    for br in (1, 128):
        q, s, qt, st = E.emb_fp8_quantize(x.cuda(), block_rows=br, transpose=True)
        for got, scale, src in ((q, s, x), (qt, st, x.t())):
            rq, rs = block_scales(src, br)
            assert torch.equal(scale.cpu(), rs) and torch.equal(bits(got), bits(rq))
            assert torch.equal(torch.isnan(got.cpu().float()), ~torch.isfinite(src))
            assert bool(torch.isfinite(scale).all() & (scale > 0).all())


def test_quantize_strided_rows_and_unaligned():
    x = torch.randn(70, 400, generator=torch.Generator().manual_seed(2)).cuda()
    for view in (x[:, :203], x[:, 3:203], x[::2, 1:130]):
        q, s, qt, st = E.emb_fp8_quantize(view, transpose=True)
        rq, rs = block_scales(view.cpu(), 1)
        assert torch.equal(s.cpu(), rs) and torch.equal(bits(q), bits(rq))
        rq, rs = block_scales(view.t().cpu(), 1)
        assert torch.equal(st.cpu(), rs) and torch.equal(bits(qt), bits(rq))


def operands(m, n, k, a_rows, b_rows, seed=0):
    g = torch.Generator().manual_seed(seed + m + 3 * n + 7 * k)
    a = torch.randn(m, k, generator=g) * torch.exp(torch.randn(m, 1, generator=g))
    b = torch.randn(n, k, generator=g) * torch.exp(torch.randn(n, 1, generator=g)) / max(k, 1) ** 0.5
    (a, sa), (b, sb) = E.emb_fp8_quantize(a.cuda(), a_rows), E.emb_fp8_quantize(b.cuda(), b_rows)
    return a, sa, b, sb


def check(out, a, sa, b, sb, bias=None):
    A, B = dequant64(a.cpu(), sa.cpu()).cuda(), dequant64(b.cpu(), sb.cpu()).cuda()
    ref, size = A @ B.t(), A.abs() @ B.abs().t()
    if bias is not None:
        ref, size = ref + bias.double(), size + bias.double().abs()
    close("out", out, ref, size, 256 + -(-a.shape[1] // 128) + 4)
    assert E.emb_check_op_flag() == 0


SHAPES = [(1, 1, 1), (1, 64, 128), (1, 333, 1000), (2, 128, 64), (3, 1024, 4096), (5, 700, 8192), (8, 96, 200), (9, 40, 300), (16, 256, 512),
          (17, 129, 130), (64, 64, 64), (100, 512, 4096), (127, 255, 129), (128, 256, 128), (128, 128, 1024), (129, 257, 385),
          (200, 1000, 16384), (256, 512, 256), (1000, 300, 1664), (1024, 1664, 2048), (2500, 96, 333), (4096, 640, 768),
          (40, 2500, 16), (300, 20, 5000), (1, 10001, 300), (1, 9729, 2100), (2, 9800, 1100), (2, 4100, 10000), (10001, 70, 300),
          (1300, 452, 692), (3000, 1293, 140)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("b_rows,out", [(128, BF16), (1, F32)])
def test_matmul(m, n, k, b_rows, out):
    a, sa, b, sb = operands(m, n, k, 1, b_rows)
    bias = torch.randn(n, generator=torch.Generator().manual_seed(n)).cuda() if out == BF16 else None
    got = E.emb_fp8_matmul(a, sa, b, sb, out_dtype=out, bias=bias)
    check(got, a, sa, b, sb, bias)
    assert torch.equal(got, E.emb_fp8_matmul(a, sa, b, sb, out_dtype=out, bias=bias))


@pytest.mark.parametrize("a_rows,b_rows", [(1, 1), (1, 128), (128, 1), (128, 128)])
@pytest.mark.parametrize("m,n,k", [(7, 130, 300), (150, 200, 260), (385, 520, 640)])
def test_matmul_scale_kinds(m, n, k, a_rows, b_rows):
    a, sa, b, sb = operands(m, n, k, a_rows, b_rows, seed=1)
    for out in (F16, F32):
        check(E.emb_fp8_matmul(a, sa, b, sb, out_dtype=out), a, sa, b, sb)


def test_matmul_strided_operands_and_output():
    m, n, k = 150, 270, 400
    a, sa, b, sb = operands(m, n, k, 1, 128, seed=2)
    wide = torch.zeros(m, 640, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    wide.view(torch.uint8)[:, :k] = a.view(torch.uint8)
    for dtype, width in ((BF16, 300), (F32, 271), (F16, 333)):
        for mm in (m, 3):
            hold = torch.full((mm, width), 7.0, dtype=dtype, device="cuda")
            out = hold[:, 1:1 + n] if width > n + 1 else hold[:, :n]
            E.emb_fp8_matmul(wide[:mm, :k], sa[:, :mm].contiguous(), b, sb, out=out)
            check(out, a[:mm], sa[:, :mm], b, sb)
            out.fill_(7.0)
            assert bool((hold == 7.0).all())      # nothing beside the output was written


def test_matmul_empty_and_nan():
    dev = dict(device="cuda")
    e = lambda r, c: torch.zeros(r, -(-c // 16) * 16, dtype=torch.uint8, **dev).view(torch.float8_e4m3fn)[:, :c]  # noqa: E731
    bias = torch.randn(6, **dev)
    out = E.emb_fp8_matmul(e(4, 0), torch.zeros(0, 4, **dev), e(6, 0), torch.zeros(0, 6, **dev), bias=bias, out_dtype=F32)
    assert torch.equal(out, bias.expand(4, 6))
    assert E.emb_fp8_matmul(e(0, 32), torch.zeros(1, 0, **dev), e(6, 32), torch.ones(1, 6, **dev)).shape == (0, 6)
    for m in (2, 40):
        x, w = torch.randn(m, 500), torch.randn(70, 500)
        x[1, 450] = float("nan")
        w[5, 2] = float("inf")
        (a, sa), (b, sb) = E.emb_fp8_quantize(x.cuda()), E.emb_fp8_quantize(w.cuda(), 128)
        out = E.emb_fp8_matmul(a, sa, b, sb, out_dtype=F32).cpu()
        bad = torch.zeros(m, 70, dtype=torch.bool)
        bad[1], bad[:, 5] = True, True
        assert torch.equal(torch.isnan(out), bad)


def test_matmul_on_another_stream_and_given_workspace():
    m, n, k = 300, 384, 4096
    a, sa, b, sb = operands(m, n, k, 1, 128, seed=4)
    want = E.emb_fp8_matmul(a, sa, b, sb)
    ws = torch.full((E.emb_fp8_matmul_workspace_size(m, n, k),), 0xFF, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [E.emb_fp8_matmul(a, sa, b, sb, workspace=ws, stream=s) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    with torch.cuda.graph(graph):
        E.emb_fp8_matmul(a, sa, b, sb, out=out, workspace=ws)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_linear_layer_gradients_against_differences():
    """A linear layer's three products from one quantisation of each tensor: its
    output, input gradient and weight gradient are those of the quantised
    operands, and agree with differences of the loss over the quantised layer
    up to the 8-bit rounding of the operands (2^-4 of each factor)."""
    g = torch.Generator().manual_seed(6)
    B, I, O = 192, 320, 256
    x, w, dy = torch.randn(B, I, generator=g), torch.randn(O, I, generator=g) / I ** 0.5, torch.randn(B, O, generator=g)
    qx, sx, qxt, sxt = E.emb_fp8_quantize(x.cuda(), 1, transpose=True)
    qw, sw, qwt, swt = E.emb_fp8_quantize(w.cuda(), 128, transpose=True)
    qd, sd, qdt, sdt = E.emb_fp8_quantize(dy.cuda(), 1, transpose=True)
    y = E.emb_fp8_matmul(qx, sx, qw, sw, out_dtype=F32)
    dx = E.emb_fp8_matmul(qd, sd, qwt, swt, out_dtype=F32)
    dw = E.emb_fp8_matmul(qdt, sdt, qxt, sxt, out_dtype=F32)
    check(y, qx, sx, qw, sw)
    check(dx, qd, sd, qwt, swt)
    check(dw, qdt, sdt, qxt, sxt)
    loss = lambda X, W: float((dy.double() * (X @ W.t())).sum())  # noqa: E731
    for got, base, other, at in ((dx, x, w, 0), (dw, w, x, 1)):
        v = torch.randn(base.shape, generator=g).double()
        up, down = base.double() + 1e-3 * v, base.double() - 1e-3 * v
        slope = (loss(up, w.double()) - loss(down, w.double()) if at == 0 else loss(x.double(), up) - loss(x.double(), down)) / 2e-3
        mine = float((got.cpu().double() * v).sum())
        terms = (dy.double().abs() @ w.double().abs() if at == 0 else dy.double().abs().t() @ x.double().abs()) * v.abs()
        assert abs(mine - slope) <= (2 * 2.0 ** -4 + 2.0 ** -8) * float(terms.sum()), (mine, slope)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("run", [4, 8, 64])
def test_quantize_scale_beside_runs_of_non_finite_values(run, block_rows, dtype):
    """Values that are not finite leave their block's scale to the finite ones, also
    where whole groups of neighbours are of that kind (a pooled row with one
    diverged slot), on and off the groups' boundaries, along rows and columns."""
    g = torch.Generator().manual_seed(run)
    x = torch.randn(260, 400, generator=g)
    for i, bad in enumerate((float("nan"), float("inf"), -float("inf"))):
        for j, at in enumerate((0, 4, 61, 128, 129, 190)):
            x[3 * j + i, at:at + run] = bad
            x[128 + at // 3:128 + at // 3 + run, 20 * i + j + 200] = bad
    x[40, 128:256] = float("nan")       # a block with nothing finite at all
    x[41, :128] = float("inf")
    x = x.to(dtype)
    q, s, qt, st = E.emb_fp8_quantize(x.cuda(), block_rows=block_rows, transpose=True)
    for got, scale, src in ((q, s, x), (qt, st, x.t())):
        rq, rs = block_scales(src, block_rows)
        assert torch.equal(scale.cpu(), rs)
        assert torch.equal(bits(got), bits(rq))
    q1, s1 = E.emb_fp8_quantize(x.cuda(), block_rows=block_rows)
    assert torch.equal(bits(q1), bits(q)) and torch.equal(s1, s)


@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("m,n,k", [(300, 512, 5120), (5000, 1100, 640), (20_011, 400, 300), (40_003, 40, 300)])
def test_a_wait_that_runs_out(m, n, k, b_rows):
    """Each warp that issues work loses its wait at the first step, while the ring of
    stages fills, and later, or the block is told to stop when the last loads are on
    their way: the product ends, raises its flag once, and leaves the GPU fit for the
    next product, which is right."""
    a, sa, b, sb = operands(m, n, k, 1, b_rows, seed=9)
    want = E.emb_fp8_matmul(a, sa, b, sb)
    check(want, a, sa, b, sb)
    steps = -(-k // 128)
    try:
        for role in ("load", "product", "scales", "other"):
            for step in (0, 1, 2, min(steps - 1, 6)):
                E.emb_debug_lose_op_wait(role, step)
                E.emb_fp8_matmul(a, sa, b, sb)
                E.emb_debug_lose_op_wait(None)
                assert E.emb_check_op_flag() == E.EMB_FLAG_OP_TIMEOUT, (role, step)
                assert E.emb_check_op_flag() == 0
                assert torch.equal(E.emb_fp8_matmul(a, sa, b, sb), want), (role, step)
                assert E.emb_check_op_flag() == 0
    finally:
        E.emb_debug_lose_op_wait(None)
    one = E.emb_fp8_matmul(a[:1], sa[:, :1].contiguous(), b, sb)
    E.emb_debug_lose_op_wait("load", 0)       # a single row waits for nothing
    try:
        assert torch.equal(E.emb_fp8_matmul(a[:1], sa[:, :1].contiguous(), b, sb), one) and E.emb_check_op_flag() == 0
    finally:
        E.emb_debug_lose_op_wait(None)


def test_flag_of_another_stream_is_reported_once():
    """Products that give up on a side stream while checks run on this one: each of
    them is reported, by a check beside it or by the one after it."""
    a, sa, b, sb = operands(300, 512, 1024, 1, 128, seed=11)
    E.emb_fp8_matmul(a, sa, b, sb)
    ws = torch.empty(E.emb_fp8_matmul_workspace_size(300, 512, 1024), dtype=torch.uint8, device="cuda")
    out = torch.empty(300, 512, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(100):
        E.emb_debug_lose_op_wait("product", 1)
        E.emb_fp8_matmul(a, sa, b, sb, out=out, workspace=ws, stream=s)
        E.emb_debug_lose_op_wait(None)
        beside = E.emb_check_op_flag()
        s.synchronize()
        assert beside | E.emb_check_op_flag(s) == E.EMB_FLAG_OP_TIMEOUT
        assert E.emb_check_op_flag() == 0


def test_flag_of_a_fresh_process():
    """The check as the first CUDA call of a process."""
    import os
    import subprocess
    import sys
    code = "import sparse_ctr_embedding_gb300 as E; assert E.emb_check_op_flag() == 0"
    subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(os.path.dirname(E.__file__)), check=True, timeout=300)


def test_linear_layer_gradients_against_differences_as_a_whole():
    """The input and the weight gradient of a quantised layer against central
    differences of the 64-bit loss <dy, x w^T>, every element of a sample: the loss
    is linear in each, so the differences are its derivatives up to 64-bit
    rounding.  Operands are rounded by at most 2^-4 of themselves, a part of one
    side independent from element to element, so the differences' norm stays within
    a tenth of the gradient's (a zero or negated gradient is off by 1 and by 2)."""
    g = torch.Generator().manual_seed(7)
    B, I, O = 96, 136, 80
    x, w, dy = torch.randn(B, I, generator=g), torch.randn(O, I, generator=g) / I ** 0.5, torch.randn(B, O, generator=g)
    _, _, qxt, sxt = E.emb_fp8_quantize(x.cuda(), 1, transpose=True)
    _, _, qwt, swt = E.emb_fp8_quantize(w.cuda(), 128, transpose=True)
    qd, sd, qdt, sdt = E.emb_fp8_quantize(dy.cuda(), 1, transpose=True)
    dx = E.emb_fp8_matmul(qd, sd, qwt, swt, out_dtype=F32).cpu().double()
    dw = E.emb_fp8_matmul(qdt, sdt, qxt, sxt, out_dtype=F32).cpu().double()
    X, Wt, D = x.double(), w.double(), dy.double()
    loss = lambda X, Wt: (D * (X @ Wt.t())).sum()  # noqa: E731
    for got, base, of in ((dx, X, lambda z: loss(z, Wt)), (dw, Wt, lambda z: loss(X, z))):
        at = torch.randperm(base.numel(), generator=g)[:400]
        slope = torch.empty(400, dtype=torch.float64)
        for i, j in enumerate(at.tolist()):
            up, down = base.clone(), base.clone()
            up.view(-1)[j] += 0.5
            down.view(-1)[j] -= 0.5
            slope[i] = of(up) - of(down)
        mine = got.reshape(-1)[at]
        assert float((mine - slope).norm() / slope.norm()) < 0.1


@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("out,wide", [(BF16, True), (F32, False)])
@pytest.mark.parametrize("m,n,k,bn", [(10_001, 1100, 300, 256), (20_011, 400, 640, 256), (5000, 1100, 300, 128), (2500, 2333, 640, 128),
                                      (40_003, 40, 300, 64), (40_003, 64, 1100, 64)])
def test_matmul_of_several_tiles_a_block(m, n, k, bn, out, wide, b_rows):
    """Whole tiles, three or more to a block, of each width: stages, scales and
    accumulators go on from tile to tile, and a tile's output is stored while the next
    one's products run.  Every element; rows of the output on and off 32 bytes."""
    cols, tiles, blocks, steps = E.emb_debug_fp8_matmul_plan(m, n, k)
    assert cols == bn and steps == 0 and tiles > 2 * blocks      # else this test has lost its subject
    a, sa, b, sb = operands(m, n, k, 1, b_rows, seed=12)
    bias = torch.randn(n, generator=torch.Generator().manual_seed(n)).cuda()
    ld = -(-n // 16) * 16 if wide else n | 1
    hold = torch.full((m, ld), 7.0, dtype=out, device="cuda")
    got = E.emb_fp8_matmul(a, sa, b, sb, bias=bias, out=hold[:, :n])
    check(got, a, sa, b, sb, bias)
    assert bool((hold[:, n:] == 7.0).all())
