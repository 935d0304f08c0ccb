"""Arrays whose element numbers pass 2^31 and 2^32: the last rows against the plain forms."""
import pytest
import torch

import sparse_ctr_embedding_gb300 as E
from dense_ref import adamw32, block_scales, close, dequant64, norm64, norm_size

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    E.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def noise(rows, dim, dtype):
    """Cheap distinct values: no second array of this size."""
    t = torch.empty(rows, dim, dtype=dtype, device="cuda")
    for r in range(0, rows, 65536):
        t[r:r + 65536] = torch.randn(min(65536, rows - r), dim, device="cuda", dtype=dtype)
    return t


def test_norm_rows_past_2_to_32_elements():
    rows, dim = 530_000, 8192
    x = noise(rows, dim, BF16)
    y, h, st = E.emb_norm_gate_fwd(x, None, eps=1e-5)
    for part in (slice(0, 3), slice(rows - 3, rows), slice(262_143, 262_146)):
        x64 = x[part].cpu().double()
        close("h", h[part], norm64(x64, None, None, False, 1e-5), norm_size(x64, None, None, False, 1e-5), 40)
    w = torch.ones(dim, device="cuda")
    d = E.emb_norm_gate_bwd(None, h, x, None, None, st, w_pre=w)
    r = slice(rows - 2, rows)
    x64, h64, s = x[r].cpu().double(), h[r].cpu().double(), st[r, 3:].cpu().double()
    hat = x64 * s
    want = s * (h64 - hat * (h64 * hat).mean(1, keepdim=True))
    size = s * (h64.abs() + hat.abs() * (h64 * hat).abs().mean(1, keepdim=True))
    close("dx", d["dx"][r], want, size, 128)
    # dw_pre = sum h * hat, over all rows
    ref = torch.zeros(dim, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    for i in range(0, rows, 65536):
        p = h[i:i + 65536].double() * (x[i:i + 65536].double() * st[i:i + 65536, 3:].double())
        ref += p.sum(0)
        mag += p.abs().sum(0)
    # rows / 152 teams at most in a row, then the teams: 4000 sequential roundings bound both
    close("dw_pre", d["dw_pre"], ref, mag, 4000 + 128)


def test_codes_and_product_past_2_to_32_bytes():
    m, n, k = 530_000, 72, 8192
    x = noise(m, k, BF16)
    q, s = E.emb_fp8_quantize(x)
    for part in (slice(0, 2), slice(m - 2, m)):
        rq, rs = block_scales(x[part].cpu(), 1)
        assert torch.equal(q[part].cpu().view(torch.uint8), rq.view(torch.uint8)) and torch.equal(s[:, part].cpu(), rs)
    w, ws = E.emb_fp8_quantize(torch.randn(n, k, device="cuda"), 128)
    out = E.emb_fp8_matmul(q, s, w, ws, out_dtype=F32)
    assert E.emb_check_op_flag() == 0
    B = dequant64(w.cpu(), ws.cpu())
    for part in (slice(0, 5), slice(262_140, 262_150), slice(m - 5, m)):
        A = dequant64(q[part].cpu(), s[:, part].cpu())
        close("out", out[part], A @ B.t(), A.abs() @ B.abs().t(), 256 + k // 128 + 4)
    wide = torch.empty(m, 8200, dtype=BF16, device="cuda")[:, 64:64 + n]       # output rows past 2^32 elements
    E.emb_fp8_matmul(q, s, w, ws, out=wide)
    assert torch.equal(wide[m - 300:], out[m - 300:].to(BF16))


def test_adamw_of_a_tensor_past_2_to_31_elements():
    n = (1 << 31) + 70_001
    p = torch.empty(n, dtype=BF16, device="cuda").fill_(0.5)
    g = torch.empty(n, dtype=BF16, device="cuda").fill_(0.25)
    g[-1000:] = torch.randn(1000, device="cuda").to(BF16)
    tail = g[-1000:].cpu()
    opt = E.AdamW([p], lr=1e-2, weight_decay=0.05, state="q8", seed=3)
    opt.step([g])
    w, m, _, _ = adamw32(torch.full((1000,), 0.5), tail, torch.zeros(1000), None, torch.zeros(1000), (1e-2, 0.9, 0.999, 1e-8, 0.05, 1), True)
    assert torch.equal(p[-1000:].cpu(), w.to(BF16))
    assert bool((p[:1000] == p[n // 2:n // 2 + 1000]).all())
    # the last block's first moments stand for m: one code apart at most (an eighth of the value, or 2^-9 of the scale)
    scale = float(opt.arena["m_scale"][(n - 1) // 256])
    count = (n - 1) % 256 + 1
    got = opt.arena["m"][n - count:n].cpu().float() * scale
    assert bool(((got - m[-count:]).abs() <= m[-count:].abs() / 8 + scale * 2.0 ** -9).all())
