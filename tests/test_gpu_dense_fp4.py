"""The 4-bit quantiser (bit for bit), reading back (exact) and matrix product (against 64 bits)."""
import pytest
import torch

import sparse_ctr_embedding_gb300 as E
from dense_ref import close
from fp4_ref import encode, pack, tile, ulps, unpack, untile, values

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    E.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def held(q):
    """All bytes of the rows, the padding included."""
    return torch.as_strided(q, (q.shape[0], q.stride(0)), (q.stride(0), 1)).cpu()


def check_codes(q, s, src, block_rows):
    code, byte = encode(src, block_rows)
    r, c = src.shape
    known = (byte != 255).repeat_interleave(32, 1)[:, :c]          # codes of a block that is NaN mean nothing
    got = unpack(q, c)
    assert torch.equal(got[known], code[known])
    rows = held(q)
    assert rows.shape[1] % 16 == 0
    if c % 2:
        assert bool((rows[:, c // 2] >> 4 == 0).all())
    assert bool((rows[:, -(-c // 2):] == 0).all())
    assert torch.equal(s.cpu(), tile(byte))                        # zeros past the edges


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (1, 33), (2, 129), (31, 64), (127, 63), (128, 128), (129, 257), (300, 1000), (5, 4099),
                                       (1030, 16)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("block_rows", [1, 32])
def test_quantize(rows, cols, dtype, block_rows):
    g = torch.Generator().manual_seed(rows * cols)
    x = (torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))).to(dtype)
    x[0, 0] = 0.0
    q, s, qt, st = E.emb_fp4_quantize(x.cuda(), block_rows=block_rows, transpose=True)
    for got, scale, src in ((q, s, x), (qt, st, x.t())):
        check_codes(got, scale, src, block_rows)
        code, byte = encode(src, block_rows)
        want = values(code, byte)
        for back in (F32, BF16):
            assert torch.equal(E.emb_fp4_dequantize(got, scale, src.shape[1], dtype=back).cpu().double(), want)
        half = E.emb_fp4_dequantize(got, scale, src.shape[1], dtype=F16).cpu()
        assert torch.equal(half, want.to(F16))
        # half a step of the nearest codes, or what lies beyond the largest one
        err, unit = (want - src.double()).abs(), 2.0 ** (byte.repeat_interleave(32, 1)[:, :src.shape[1]].double() - 127)
        assert bool((err <= torch.maximum(src.double().abs() / 4, unit / 4)).all())
    if block_rows == 32:
        assert torch.equal(E.emb_fp4_dequantize(q, s, cols, dtype=F32), E.emb_fp4_dequantize(qt, st, rows, dtype=F32).t())
    q1, s1 = E.emb_fp4_quantize(x.cuda(), block_rows=block_rows)
    assert torch.equal(held(q1), held(q)) and torch.equal(s1, s)


@pytest.mark.parametrize("block_rows", [1, 32])
def test_quantize_every_rounding(block_rows):
    """Every code, every tie between two and what lies beside it, at exponents over the whole range."""
    marks = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0, 7.9999995])
    beside = torch.cat([marks, torch.nextafter(marks, torch.tensor(9.0)), torch.nextafter(marks, torch.tensor(-9.0))])
    v = torch.cat([beside, -beside])[:96]
    rows = torch.zeros(40, 32 * 4)
    for i in range(40):
        e = [-149, -146, -127, -126, -125, -124, -60, -3, -1, 0, 1, 2, 30, 100, 124][i % 15]
        part = v.roll(7 * i)[:31].double()
        for b in range(4):
            rows[i, 32 * b:32 * b + 31] = (part.roll(b) * 2.0 ** e).clamp(-3.4e38, 3.4e38).float()
            rows[i, 32 * b + 31] = float(min(4.0 * 2.0 ** e, 2.0 ** 127))
    if block_rows == 32:
        rows = rows[:1].expand(32, -1).clone() * torch.exp2(torch.arange(32) % 3 - 1.0)[:, None]
    q, s, qt, st = E.emb_fp4_quantize(rows.cuda(), block_rows=block_rows, transpose=True)
    check_codes(q, s, rows, block_rows)
    check_codes(qt, st, rows.t(), block_rows)
    code, byte = encode(rows, block_rows)
    assert torch.equal(E.emb_fp4_dequantize(q, s, dtype=F32).cpu().double(), values(code, byte))


@pytest.mark.parametrize("block_rows", [1, 32])
def test_quantize_special_values(block_rows):
    x = torch.randn(200, 256, generator=torch.Generator().manual_seed(1))
    x[0, :128] = 0.0
    x[1, 5], x[70, 130] = float("inf"), float("nan")
    x[2, :128] = 1e-42
    x[3, 3] = 3e38
    x[180, 255] = -float("inf")
    q, s, qt, st = E.emb_fp4_quantize(x.cuda(), block_rows=block_rows, transpose=True)
    for got, scale, src in ((q, s, x), (qt, st, x.t())):
        check_codes(got, scale, src, block_rows)
        code, byte = encode(src, block_rows)
        back = E.emb_fp4_dequantize(got, scale, src.shape[1], dtype=F32).cpu().double()
        assert torch.equal(back.nan_to_num(7.0), values(code, byte).nan_to_num(7.0))
        bad = (~torch.isfinite(src)).double()
        assert int(torch.isnan(back).sum()) >= int(bad.sum()) > 0


def test_quantize_strided_rows_unaligned_and_empty():
    g = torch.Generator().manual_seed(3)
    hold = torch.randn(70, 301, generator=g).cuda()
    for dtype in (F32, BF16, F16):
        for view in (hold.to(dtype)[:, 1:200], hold.to(dtype)[1:, 4:300], hold.to(dtype)[::2, :128]):
            q, s, qt, st = E.emb_fp4_quantize(view, transpose=True)
            check_codes(q, s, view.cpu(), 1)
            check_codes(qt, st, view.cpu().t(), 1)
            out = torch.full((view.shape[0], view.shape[1] + 5), 9.0, device="cuda")
            E.emb_fp4_dequantize(q, s, view.shape[1], out=out[:, 2:2 + view.shape[1]])
            assert torch.equal(out[:, 2:2 + view.shape[1]], E.emb_fp4_dequantize(q, s, view.shape[1], dtype=F32))
            assert bool((out[:, :2] == 9.0).all()) and bool((out[:, 2 + view.shape[1]:] == 9.0).all())
    for shape in ((0, 40), (40, 0)):
        q, s, qt, st = E.emb_fp4_quantize(torch.zeros(shape, device="cuda"), transpose=True)
        assert E.emb_fp4_dequantize(q, s, shape[1]).shape == shape and E.emb_fp4_dequantize(qt, st, shape[0]).shape == shape[::-1]


def operands(m, n, k, seed=0):
    g = torch.Generator().manual_seed(seed * 1000 + m + n + k)
    x = torch.randn(m, k, generator=g) * torch.exp(torch.randn(m, 1, generator=g))
    w = torch.randn(n, k, generator=g) * torch.exp(torch.randn(n, 1, generator=g)) / k ** 0.5
    return (*E.emb_fp4_quantize(x.cuda()), *E.emb_fp4_quantize(w.cuda()))


def matrix(q, s, cols=None):
    cols = 2 * q.shape[1] if cols is None else cols
    return values(unpack(q, cols), untile(s, q.shape[0], -(-cols // 32)))


def check(out, a, sa, b, sb, bias=None):
    A, B = matrix(a, sa).cuda(), matrix(b, sb).cuda()
    ref, size = A @ B.t(), A.abs() @ B.abs().t()
    if bias is not None:
        ref, size = ref + bias.double(), size + bias.double().abs()
    close("out", out, ref, size, ulps(2 * a.shape[1]))
    assert E.emb_check_op_flag() == 0


SHAPES = [(1, 1, 1), (1, 64, 128), (1, 333, 1000), (2, 128, 64), (3, 64, 64), (128, 128, 256), (128, 64, 64), (128, 256, 128), (3, 1024, 4096),
          (5, 700, 8192), (8, 96, 200), (9, 40, 300), (16, 256, 512), (17, 129, 130), (64, 64, 64), (100, 512, 4096), (127, 255, 129),
          (128, 128, 1024), (129, 257, 385), (200, 1000, 16384), (256, 512, 256), (1000, 300, 1664), (1024, 1664, 2048), (2500, 96, 333),
          (4096, 640, 768), (40, 2500, 16), (300, 20, 5000), (1, 10001, 300), (1, 9729, 2100), (2, 9800, 1100), (2, 4100, 10000),
          (10001, 70, 300), (1300, 452, 692), (2500, 1293, 141), (20_011, 1100, 8192), (1000, 520, 80_000)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("out", [BF16, F32])
def test_matmul(m, n, k, out):
    a, sa, b, sb = operands(m, n, k)
    bias = torch.randn(n, generator=torch.Generator().manual_seed(n)).cuda() if out == BF16 else None
    got = E.emb_fp4_matmul(a, sa, b, sb, out_dtype=out, bias=bias)
    check(got, a, sa, b, sb, bias)
    assert torch.equal(got, E.emb_fp4_matmul(a, sa, b, sb, out_dtype=out, bias=bias))


def test_matmul_strided_operands_and_output():
    m, n, k = 150, 270, 401
    a, sa, b, sb = operands(m, n, k, seed=2)
    wide = torch.full((m, 320), 0x77, dtype=torch.uint8, device="cuda")      # codes past k are not used
    wide[:, :a.shape[1]] = a
    for dtype, width in ((BF16, 300), (F32, 271), (F16, 333)):
        for mm in (m, 2, 1):
            hold = torch.full((mm, width), 7.0, dtype=dtype, device="cuda")
            out = hold[:, 1:1 + n] if width > n + 1 else hold[:, :n]
            E.emb_fp4_matmul(wide[:mm, :a.shape[1]], sa[:-(-mm // 128)].contiguous(), b, sb, out=out)
            check(out, a[:mm], sa, b, sb)
            out.fill_(7.0)
            assert bool((hold == 7.0).all())      # nothing beside the output was written


def test_matmul_scales_over_the_range():
    """Rows whose scales differ by up to 2^250 meet in products that are within float32's range."""
    g = torch.Generator().manual_seed(5)
    for m in (1, 40):
        e = torch.arange(40).double() * 6 - 120
        x = (torch.randn(40, 320, generator=g).double() * 2.0 ** e[:, None]).float()
        w = (torch.randn(40, 320, generator=g).double() * 2.0 ** -e[:, None]).float()
        for i in range(0, 40, 7):
            (a, sa), (b, sb) = E.emb_fp4_quantize(x[i:i + m].cuda()), E.emb_fp4_quantize(w[i:i + m].cuda())
            A, B = matrix(a, sa).cuda(), matrix(b, sb).cuda()
            ref, size = A @ B.t(), A.abs() @ B.abs().t()
            keep = size < 2.0 ** 126
            got = E.emb_fp4_matmul(a, sa, b, sb, out_dtype=F32)
            close("out", got[keep], ref[keep], size[keep], ulps(320))
            assert int(keep.sum()) >= 1


def test_matmul_empty_and_nan():
    dev = dict(device="cuda")
    codes = lambda r, c: torch.zeros(r, c // 2, dtype=torch.uint8, **dev)  # noqa: E731
    scales = lambda r, c: torch.zeros(-(-r // 128), -(-c // 128), 32, 4, 4, dtype=torch.uint8, **dev)  # noqa: E731
    bias = torch.randn(6, **dev)
    out = E.emb_fp4_matmul(codes(4, 0), scales(4, 0), codes(6, 0), scales(6, 0), bias=bias, out_dtype=F32)
    assert torch.equal(out, bias.expand(4, 6))
    assert E.emb_fp4_matmul(codes(0, 32), scales(0, 32), codes(6, 32), scales(6, 32)).shape == (0, 6)
    for m in (1, 2, 40):
        x, w = torch.randn(m, 500), torch.randn(70, 500)
        x[m - 1, 450] = float("nan")
        w[5, 2] = float("inf")
        (a, sa), (b, sb) = E.emb_fp4_quantize(x.cuda()), E.emb_fp4_quantize(w.cuda())
        out = E.emb_fp4_matmul(a, sa, b, sb, out_dtype=F32).cpu()
        bad = torch.zeros(m, 70, dtype=torch.bool)
        bad[m - 1], bad[:, 5] = True, True
        assert torch.equal(torch.isnan(out), bad)


def test_matmul_on_another_stream_and_in_a_graph():
    m, n, k = 300, 384, 4096
    a, sa, b, sb = operands(m, n, k, seed=4)
    want = E.emb_fp4_matmul(a, sa, b, sb)
    ws = torch.full((E.emb_fp4_matmul_workspace_size(m, n, k),), 0xFF, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [E.emb_fp4_matmul(a, sa, b, sb, workspace=ws, stream=s) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)
    graph = torch.cuda.CUDAGraph()
    out, x = torch.empty_like(want), torch.randn(m, k, device="cuda")
    back = torch.empty(m, k, device="cuda")
    with torch.cuda.graph(graph):
        E.emb_fp4_matmul(a, sa, b, sb, out=out, workspace=ws)
        q, e = E.emb_fp4_quantize(x)
        E.emb_fp4_dequantize(q, e, out=back)
    for _ in range(2):
        out.zero_()
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert torch.equal(back, E.emb_fp4_dequantize(*E.emb_fp4_quantize(x), dtype=F32))


def test_linear_layer_gradients():
    """A linear layer's three products from one quantisation of each tensor: they are
    those of the quantised operands, and the derivatives of the loss <dy, x w^T> by its
    differences over the quantised layer (linear in each operand, so exact up to rounding)."""
    g = torch.Generator().manual_seed(6)
    B, I, O = 192, 320, 256
    x, w, dy = torch.randn(B, I, generator=g), torch.randn(O, I, generator=g) / I ** 0.5, torch.randn(B, O, generator=g)
    qx, sx, qxt, sxt = E.emb_fp4_quantize(x.cuda(), 1, transpose=True)
    qw, sw, qwt, swt = E.emb_fp4_quantize(w.cuda(), 32, transpose=True)
    qd, sd, qdt, sdt = E.emb_fp4_quantize(dy.cuda(), 1, transpose=True)
    check(E.emb_fp4_matmul(qx, sx, qw, sw, out_dtype=F32), qx, sx, qw, sw)
    dx = E.emb_fp4_matmul(qd, sd, qwt, swt, out_dtype=F32)
    dw = E.emb_fp4_matmul(qdt, sdt, qxt, sxt, out_dtype=F32)
    check(dx, qd, sd, qwt, swt)
    check(dw, qdt, sdt, qxt, sxt)
    D, W = matrix(qd, sd), matrix(qw, sw)              # both orientations of w hold the same values
    loss = lambda X: (D * (X @ W.t())).sum()  # noqa: E731
    X = x.double()
    for _ in range(20):
        i, j = int(torch.randint(B, (1,), generator=g)), int(torch.randint(I, (1,), generator=g))
        up, down = X.clone(), X.clone()
        up[i, j] += 0.5
        down[i, j] -= 0.5
        slope = float(loss(up) - loss(down))
        assert abs(float(dx[i, j]) - slope) <= (ulps(O) * 2.0 ** -24 + 1e-9) * float((D.abs() @ W.abs())[i, j]) + 1e-9 * float((D * (X @ W.t())).abs().sum())
    DT, XT = matrix(qdt, sdt), matrix(qxt, sxt)
    assert float((DT.t() - dy).norm() / dy.norm()) < 0.25 and float((XT.t() - x).norm() / x.norm()) < 0.25


@pytest.mark.parametrize("m,n,k", [(300, 512, 5120), (5000, 1100, 640), (20_011, 400, 300), (40_003, 40, 300), (1024, 1664, 16384)])
def test_a_wait_that_runs_out(m, n, k):
    """Each warp that issues work loses its wait at the first step, while the ring of
    stages fills, and later, or the block is told to stop when the last loads are on
    their way: the product ends, raises its flag once, and leaves the GPU fit for the
    next product, which is right."""
    a, sa, b, sb = operands(m, n, k, seed=9)
    want = E.emb_fp4_matmul(a, sa, b, sb)
    check(want, a, sa, b, sb)
    steps = -(-k // 256)
    try:
        for role in ("load", "product", "other"):
            for step in (0, 1, min(steps - 1, 6)):
                E.emb_debug_lose_op_wait(role, step)
                E.emb_fp4_matmul(a, sa, b, sb)
                E.emb_debug_lose_op_wait(None)
                assert E.emb_check_op_flag() == E.EMB_FLAG_OP_TIMEOUT, (role, step)
                assert E.emb_check_op_flag() == 0
                assert torch.equal(E.emb_fp4_matmul(a, sa, b, sb), want), (role, step)
                assert E.emb_check_op_flag() == 0
    finally:
        E.emb_debug_lose_op_wait(None)


@pytest.mark.parametrize("out,wide", [(BF16, True), (F32, False)])
@pytest.mark.parametrize("m,n,k", [(20_011, 1100, 300), (66_000, 512, 1000), (100_001, 300, 130), (40_011, 400, 640), (40_003, 40, 300), (60_003, 64, 1100), (30_000, 200, 96)])
def test_matmul_of_several_tiles_a_block(m, n, k, out, wide):
    """Whole tiles, several to a block: stages and accumulators go on from tile to tile,
    and a tile's output is stored while the next one's products run."""
    a, sa, b, sb = operands(m, n, k, seed=12)
    bias = torch.randn(n, generator=torch.Generator().manual_seed(n)).cuda()
    ld = -(-n // 16) * 16 if wide else n | 1
    hold = torch.full((m, ld), 7.0, dtype=out, device="cuda")
    got = E.emb_fp4_matmul(a, sa, b, sb, bias=bias, out=hold[:, :n])
    check(got, a, sa, b, sb, bias)
    assert bool((hold[:, n:] == 7.0).all())


def test_plans():
    """The sizes above reach every kernel: rows, each width of a tile, pairs, whole and shared tiles."""
    seen = set()
    for m, n, k in SHAPES + [(300, 512, 5120), (5000, 1100, 640), (20_011, 400, 300), (40_003, 40, 300), (1024, 1664, 16384), (20_011, 1100, 300),
                             (66_000, 512, 1000), (100_001, 300, 130), (40_011, 400, 640), (60_003, 64, 1100), (30_000, 200, 96)]:
        cols, tiles, workers, steps, blocks = E.emb_debug_fp4_matmul_plan(m, n, k)
        seen.add((cols, blocks, steps > 0))
        assert workers <= 152 // blocks or cols == 0
    assert {(0, 1, False), (256, 2, False), (256, 2, True)} <= seen, seen
    print(seen)


@pytest.mark.parametrize("cols", [2, 31, 33, 40, 63, 129, 1000, 1007, 2078, 10_001])
def test_rows_that_end_their_tensor(cols):
    """Codes whose storage ends with the last row's last byte: products and values are those of padded rows, and
    what lies behind the row does not count."""
    g = torch.Generator().manual_seed(cols)
    w = -(-cols // 2)
    ld = -(-w // 16) * 16
    for rows in (1, 2, 3):
        x = torch.randn(rows, cols, generator=g).cuda()
        q, s = E.emb_fp4_quantize(x)
        room = torch.full((rows * ld + 64,), 0x77, dtype=torch.uint8, device="cuda")
        short = torch.empty((rows - 1) * ld + w, dtype=torch.uint8, device="cuda")     # not a byte more
        for hold in (room[:(rows - 1) * ld + w], short):
            t = hold.as_strided((rows, w), (ld, 1), hold.storage_offset())
            t.copy_(q)
            for dtype in (F32, BF16, F16):
                assert torch.equal(E.emb_fp4_dequantize(t, s, cols, dtype=dtype), E.emb_fp4_dequantize(q, s, cols, dtype=dtype))
            for n in (1, 40, 10_001 if cols < 2000 else 500):
                b, sb = E.emb_fp4_quantize(torch.randn(n, cols, generator=g).cuda() / cols ** 0.5)
                got = E.emb_fp4_matmul(t, s, b, sb, out_dtype=F32)
                assert torch.equal(got, E.emb_fp4_matmul(q, s, b, sb, out_dtype=F32))
                check(got, q, s, b, sb)
                back = E.emb_fp4_matmul(b, sb, t, s, out_dtype=F32)
                assert torch.equal(back, E.emb_fp4_matmul(b, sb, q, s, out_dtype=F32))
                check(back, b, sb, q, s)
    one = E.emb_fp4_quantize(torch.randn(1, cols, generator=g).cuda())
    clone = one[0].clone(memory_format=torch.contiguous_format)
    assert clone.untyped_storage().nbytes() == w and torch.equal(E.emb_fp4_dequantize(clone, one[1], cols), E.emb_fp4_dequantize(*one, cols))


# (columns of a tile or 0, blocks of a worker, steps shared out) of every product, and sizes that reach it on a GPU of 152 SMs
PLANS = {(0, 1, False): [(1, 1024, 8190), (2, 777, 1002)],
         (64, 1, False): [(123, 835, 1490), (307, 1233, 622)],
         (64, 1, True): [(64, 1024, 8192), (570, 81, 5426)],
         (128, 1, False): [(1024, 1664, 16384), (1471, 3423, 1602)],
         (128, 1, True): [(581, 210, 33658), (9, 67, 39406)],
         (256, 1, False): [(2051, 3657, 4846), (1813, 1301, 322)],
         (256, 1, True): [(50, 8734, 15630), (7, 2197, 32284), (1303, 910, 22926)],
         (256, 2, False): [(20_011, 1024, 8192), (1843, 1358, 7090)],
         (256, 2, True): [(133, 3037, 14134), (1000, 520, 80_000)]}


def plan_of(m, n, k):
    cols, _, _, steps, blocks = E.emb_debug_fp4_matmul_plan(m, n, k)
    return cols, blocks, steps > 0


def sizes_of(plan, count):
    """Sizes that this GPU runs by this plan: those above where they do, else the first of a seeded search that do."""
    found = [s for s in sum(PLANS.values(), []) if plan_of(*s) == plan]
    g = torch.Generator().manual_seed(1)
    for u in torch.rand(100_000, 3, generator=g, dtype=torch.float64).tolist() if len(found) < count else ():
        m, n, k = int(60_000 ** u[0]), int(32 * 300 ** u[1]), 2 * int(16 * 1000 ** u[2])
        if m * k <= 8e7 and n * k <= 8e7 and m * n * k <= 1.2e11 and plan_of(m, n, k) == plan:
            found.append((m, n, k))
            if len(found) >= count:
                break
    assert len(found) >= count, plan
    return found


@pytest.mark.parametrize("plan", PLANS, ids=str)
def test_every_plan(plan):
    """Each kernel and way to cut the work, into aligned rows of output (whole vectors) and others, in all three types."""
    for m, n, k in sizes_of(plan, 2):
        a, sa, b, sb = operands(m, n, k, seed=21)
        bias = torch.randn(n, generator=torch.Generator().manual_seed(n)).cuda()
        A, B = matrix(a, sa).cuda(), matrix(b, sb).cuda()
        ref, size = A @ B.t() + bias.double(), A.abs() @ B.abs().t() + bias.double().abs()
        del A, B
        for dtype in (BF16, F32, F16):
            got = []
            for ld in (-(-n // 16) * 16, n | 1):
                hold = torch.full((m, ld), 7.0, dtype=dtype, device="cuda")
                out = E.emb_fp4_matmul(a, sa, b, sb, bias=bias, out=hold[:, :n])
                close("out", out, ref, size, ulps(k))
                assert bool((hold[:, n:] == 7.0).all())
                got.append(out)
            assert torch.equal(*got), (m, n, k, dtype)
        assert E.emb_check_op_flag() == 0


@pytest.mark.parametrize("plan", [p for p in PLANS if p[0]], ids=str)
def test_a_wait_of_every_plan_that_runs_out(plan):
    """As test_a_wait_that_runs_out, for pairs of SMs and each width of a tile, whole and shared."""
    m, n, k = sizes_of(plan, 1)[0]
    a, sa, b, sb = operands(m, n, k, seed=22)
    want = E.emb_fp4_matmul(a, sa, b, sb)
    check(want, a, sa, b, sb)
    steps = E.emb_debug_fp4_matmul_plan(m, n, k)[3] or -(-k // 256)        # that a worker takes at least
    try:
        for role in ("load", "product", "other"):
            for step in sorted({0, min(steps - 1, 1), min(steps - 1, 6)}):
                E.emb_debug_lose_op_wait(role, step)
                E.emb_fp4_matmul(a, sa, b, sb)
                E.emb_debug_lose_op_wait(None)
                assert E.emb_check_op_flag() == E.EMB_FLAG_OP_TIMEOUT, (role, step)
                assert E.emb_check_op_flag() == 0
                assert torch.equal(E.emb_fp4_matmul(a, sa, b, sb), want), (role, step)
                assert E.emb_check_op_flag() == 0
    finally:
        E.emb_debug_lose_op_wait(None)
