"""Measured cases of the tower's 4-bit layers, its matrix optimizer and its plain embeddings.

Beside the 8-bit layers, the norms and AdamW, a tower on the pooled embeddings
runs: linear layers in microscaled 4-bit codes (quantiser, reading back,
product), Muon for its matrices, and embeddings of small vocabularies or of
item sequences that are kept row by row (lookup with a scale, gradient by sorted
tokens).  Each case is one pass through one of them.  Where `own` is false `run`
computes it from elementary torch operations in float32; where it is true it
calls the library.
"""
import math

import torch

own = False

BLOCK = 32             # elements that share one power-of-two scale
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i32": torch.int32, "i64": torch.int64}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "i32": 4, "i64": 8}
NS = (3.4445, -4.7750, 2.0315)   # coefficients of one Newton-Schulz step
NS_STEPS = 5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # pooled output of 100 slots x 32 for a whole training batch: codes for the forward and for the weight gradient
        {"name": "quantize4_pooled", "op": "quantize", "rows": 65536, "cols": 3200, "type": "f32", "block_rows": 1,
         "back": "bf16"},
        # a small weight with scales shared by both orientations, odd number of rows
        {"name": "quantize4_weight", "op": "quantize", "rows": 1001, "cols": 1984, "type": "bf16", "block_rows": 32,
         "back": "f32"},
        # scoring one sample: the first layer over 64 slots x 128, bound by reading the weight
        {"name": "matmul4_one_row", "op": "matmul", "m": 1, "n": 1024, "k": 8192, "out": "bf16", "bias": True},
        # weight gradient of the first layer over 26 slots x 64: the batch is the long axis
        {"name": "matmul4_weight_grad", "op": "matmul", "m": 1024, "n": 1664, "k": 16384, "out": "f32", "bias": False},
        # forward of the first layer over 64 slots x 128 for the largest training batch
        {"name": "matmul4_fwd_large", "op": "matmul", "m": 131072, "n": 1024, "k": 8192, "out": "bf16", "bias": True},
        # a small tower's matrices: latency counts
        {"name": "muon_small", "op": "muon", "shapes": "256x512,128x256,64x128", "param": "bf16", "grad": "bf16",
         "products": "half"},
        # the tower over 64 slots x 128, float32 weights, updates to float32's accuracy
        {"name": "muon_tower_f32", "op": "muon", "shapes": "1024x8192,1024x1024,512x1024,256x512", "param": "f32",
         "grad": "bf16", "products": "split"},
        # wide square layers, tall and odd ones among them: bound by the products
        {"name": "muon_large", "op": "muon", "shapes": "4096x4096,4096x2048,2048x4096,1664x1001,333x1000",
         "param": "bf16", "grad": "f32", "products": "half"},
        # one sample with a history of 50 items being scored: pure latency
        {"name": "tokens_fwd_one", "op": "tokens_fwd", "n": 50, "vocab": 100000, "dim": 64, "weight": "f16",
         "out": "bf16", "token": "i64", "pad": 0.0},
        # item sequences of a training batch (16,384 samples, 100 items at most), rows padded
        {"name": "tokens_fwd_batch", "op": "tokens_fwd", "n": 1638400, "vocab": 1000000, "dim": 128, "weight": "f32",
         "out": "bf16", "token": "i64", "pad": 0.3},
        # their gradient, long-tailed ids
        {"name": "tokens_bwd_batch", "op": "tokens_bwd", "n": 1638400, "vocab": 1000000, "dim": 128, "weight": "f32",
         "grad": "bf16", "token": "i64", "pad": 0.3},
        # a position feature: few tokens, each of them thousands of times
        {"name": "tokens_bwd_position", "op": "tokens_bwd", "n": 409600, "vocab": 201, "dim": 64, "weight": "f32",
         "grad": "f32", "token": "i32", "pad": 0.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "muon", "tokens_fwd", "tokens_bwd"])
    if op == "quantize":
        cols = _log_int(rng, 32, 8192)
        if rng.random() < 0.5:
            cols = max(32, cols // 32 * 32)
        rows = _log_int(rng, 1, min(131072, 65536 * 3200 // cols))
        return {"op": op, "rows": rows, "cols": cols, "type": rng.choice(["f32", "bf16", "f16"]),
                "block_rows": rng.choice([1, 32]), "back": rng.choice(["bf16", "f32"])}
    if op == "matmul":
        m, n, k = _log_int(rng, 1, 131072), _log_int(rng, 32, 2048), _log_int(rng, 32, 16384)
        if rng.random() < 0.6:
            n, k = max(32, n // 32 * 32), max(32, k // 32 * 32)
        m = max(1, min(m, 131072 * 8192 // k, 131072 * 8192 * 1024 // (n * k)))
        return {"op": op, "m": m, "n": n, "k": k, "out": rng.choice(["bf16", "f32", "f16"]), "bias": bool(rng.randrange(2))}
    if op == "muon":
        shapes, left = [], 1e11
        for _ in range(rng.randrange(1, 7)):
            r, c = _log_int(rng, 16, 4096), _log_int(rng, 16, 8192)
            if rng.random() < 0.5:
                r, c = max(16, r // 16 * 16), max(16, c // 16 * 16)
            c = min(c, int(1e11 / r ** 2)) if r <= c else c
            if rng.random() < 0.3:
                r, c = c, r
            cost = min(r, c) ** 2 * max(r, c)
            if cost <= left:
                shapes.append((r, c))
                left -= cost
        param = rng.choice(["f32", "bf16", "f16"])
        return {"op": op, "shapes": ",".join("%dx%d" % s for s in shapes), "param": param,
                "grad": rng.choice(["f32", "bf16"]), "products": "split" if param == "f32" else "half"}
    vocab, dim = _log_int(rng, 10, 2000000), _log_int(rng, 4, 1024)
    if rng.random() < 0.7:
        dim = max(4, dim // 4 * 4)
    vocab = min(vocab, 128000000 // dim)
    n = _log_int(rng, 1, min(1638400, 209715200 // dim))
    case = {"op": op, "n": n, "vocab": vocab, "dim": dim, "weight": rng.choice(["f32", "bf16", "f16"]),
            "token": rng.choice(["i32", "i64"]), "pad": rng.choice([0.0, 0.3])}
    case["out" if op == "tokens_fwd" else "grad"] = rng.choice(["f32", "bf16", "f16"])
    return case


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def work(case):
    op = case["op"]
    if op == "quantize":    # x in; codes, scales and the values read back out, in both orientations
        n = case["rows"] * case["cols"]
        return {"bytes": n * (BYTES[case["type"]] + 2 * BYTES[case["back"]]) + 2 * (n // 2 + n // BLOCK), "flops": 4 * n}
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * (k // 2 + k // BLOCK) + m * n * BYTES[case["out"]] + (4 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    if op == "muon":
        sizes = [(min(s), max(s)) for s in _shapes(case)]
        return {"bytes": sum(s * w for s, w in sizes) * (2 * BYTES[case["param"]] + BYTES[case["grad"]] + 8),
                "flops": sum(NS_STEPS * (3 * s * s * w + s ** 3) for s, w in sizes)}
    n, v, d = case["n"], case["vocab"], case["dim"]
    if op == "tokens_fwd":  # a row of the weight is read once, however many tokens name it
        return {"bytes": min(n, v) * d * BYTES[case["weight"]] + n * (d * BYTES[case["out"]] + BYTES[case["token"]]), "flops": n * d}
    return {"bytes": n * (d * BYTES[case["grad"]] + BYTES[case["token"]]) + v * d * BYTES[case["weight"]], "flops": 2 * n * d}


# ------------------------------------------------------------------ inputs

def _tiled(e):
    """Scale bytes [rows, ceil(k/32)] in the order the tensor cores read them: tiles of 128 rows x 4 blocks, in a tile
    [row % 32][row / 32][block]; zeros past the edges."""
    r, b = e.shape
    e = torch.nn.functional.pad(e, (0, -b % 4, 0, -r % 128))
    return e.view(e.shape[0] // 128, 4, 32, e.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous()


def _codes(rows, cols, std, gen):
    """A quantised matrix as the quantiser lays it out: two codes a byte in rows of 16-byte multiples, tiled scales."""
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    x *= std * torch.exp(torch.randn(rows, 1, device="cuda", generator=gen))    # samples and channels differ in size
    value, e = _quantize(x, 1)
    del x
    mag = value.abs()
    code = torch.where(mag < 2, 2 * mag, torch.where(mag < 4, mag + 2, 4 + mag / 2)).floor().clamp_max(7).to(torch.uint8)
    del mag
    code = code + (value < 0) * 8
    code = torch.nn.functional.pad(code, (0, cols % 2))
    held = torch.zeros(rows, -(-cols // 32) * 16, dtype=torch.uint8, device="cuda")[:, :-(-cols // 2)]
    held.copy_(code[:, 0::2] + 16 * code[:, 1::2])
    return held, _tiled(e)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]

    def normal(*shape, std=1.0, t="f32"):
        return (torch.randn(*shape, device="cuda", generator=g) * std).to(TYPES[t])

    if op == "quantize":
        x = normal(case["rows"], case["cols"], std=0.05) * torch.exp(normal(case["rows"], 1))
        return {"case": case, "x": x.to(TYPES[case["type"]])}
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        s = {"case": case, "bias": normal(n) if case["bias"] else None}
        s["a"], s["sa"] = _codes(m, k, 1.0, g)
        s["b"], s["sb"] = _codes(n, k, k ** -0.5, g)
        if own:
            import sparse_ctr_embedding_gb300 as E
            s["workspace"] = torch.empty(E.emb_fp4_matmul_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")
        return s
    if op == "muon":
        s = {"case": case, "p": [], "grad": [], "m": [], "lr": 1e-3, "momentum": 0.95, "weight_decay": 0.1}
        for r, c in _shapes(case):
            # gradients have a few strong directions and a broad rest; the momentum is an average of such
            k = max(1, min(r, c) // 16)
            strong = [normal(r, k) @ normal(k, c) * (1e-3 / k ** 0.5) for _ in range(2)]
            s["p"].append(normal(r, c, std=c ** -0.5, t=case["param"]))
            s["grad"].append((strong[0] + strong[1] + normal(r, c, std=1e-3)).to(TYPES[case["grad"]]))
            s["m"].append(strong[0] + normal(r, c, std=3e-4))
        if own:   # the optimizer object that a program keeps, on these buffers
            import sparse_ctr_embedding_gb300 as E
            s["opt"] = E.Muon(s["p"], lr=s["lr"], momentum=s["momentum"], weight_decay=s["weight_decay"],
                              products=case["products"])
            s["opt"].load_state(s["m"])
            s["m"] = s["opt"].m
        return s
    n, v, d = case["n"], case["vocab"], case["dim"]
    rank = torch.rand(n, dtype=torch.float64, device="cuda", generator=g)
    if v > 1000:     # long-tailed: the k-th most frequent id comes about 1/k as often; its rows lie anywhere
        rank = (float(v) ** rank - 1.0).long().clamp(0, v - 1)
        ids = (rank * 2654435761 + 12345) % v
    else:
        ids = (rank * v).long().clamp(0, v - 1)
    if case["pad"]:
        ids = torch.where(torch.rand(n, device="cuda", generator=g) < case["pad"], -1, ids)
    s = {"case": case, "tokens": ids.to(TYPES[case["token"]]), "scale": d ** 0.5}
    if op == "tokens_fwd":
        s["weight"] = normal(v, d, std=d ** -0.5, t=case["weight"])
    else:
        s["grad"] = normal(n, d, std=1e-2, t=case["grad"])
        if own:
            import sparse_ctr_embedding_gb300 as E
            s["workspace"] = torch.empty(E.emb_token_bwd_workspace_size(n, v, d), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _power(byte):
    """2^(byte - 127) in float32, exactly: the smallest is a denormal number, 255 stands for NaN."""
    bits = torch.where(byte == 0, 0x400000, torch.where(byte == 255, 0x7fc00000, byte.to(torch.int32) << 23))
    return bits.view(torch.float32)


def _quantize(x, block_rows):
    """Values of the codes of a float32 matrix (without their scale), and scale bytes [rows, ceil(cols/32)]."""
    r, c = x.shape
    t = torch.nn.functional.pad(x, (0, -c % BLOCK, 0, -r % block_rows))
    t = t.view(t.shape[0] // block_rows, block_rows, t.shape[1] // BLOCK, BLOCK)
    amax = t.abs().amax((1, 3), keepdim=True)
    e = (torch.frexp(amax)[1] - 3 + 127).clamp(0, 254)           # floor(log2 amax) - 2
    e = torch.where(amax == 0, 0, torch.where(amax < math.inf, e, 255))
    v = t * _power((254 - e).clamp_min(0))                       # by a power of two: exact
    mag = v.abs()
    step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0))
    v = torch.sign(v) * (torch.round(mag / step) * step).clamp_max(6.0)
    e = e.to(torch.uint8)[:, 0, :, 0].repeat_interleave(block_rows, 0)[:r]
    return v.reshape(-1, t.shape[2] * BLOCK)[:r, :c], e


def _values(value, e, t):
    return (value * _power(e).repeat_interleave(BLOCK, 1)[:, :value.shape[1]]).to(TYPES[t])


def _decode(q, s):
    """The float32 matrix that packed codes and tiled scales stand for."""
    r, c = q.shape[0], 2 * q.shape[1]
    mags = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    table = torch.cat([mags, -mags])
    pairs = torch.stack([table.repeat(16), table.repeat_interleave(16)], 1)    # by byte: low code, high code
    e = s.permute(0, 3, 2, 1, 4).reshape(s.shape[0] * 128, -1)[:r]
    x = pairs[q.reshape(-1).int()].view(r, c)
    return x * _power(e).repeat_interleave(BLOCK, 1)[:, :c]


def _orthogonal(u):
    a, b, c = NS
    x = u / (torch.sqrt((u * u).sum()) + 1e-7)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t()
    for _ in range(NS_STEPS):
        g = x @ x.t()
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.t() if tall else x


def _muon(s):
    beta = s["momentum"]
    for p, g, m in zip(s["p"], s["grad"], s["m"]):
        g = g.float()
        m.copy_(beta * m + (1.0 - beta) * g)
        x = _orthogonal((1.0 - beta) * g + beta * m)
        scale = 0.2 * max(p.shape) ** 0.5
        p.copy_(p.float() * (1.0 - s["lr"] * s["weight_decay"]) - (s["lr"] * scale) * x)
    return {"p": s["p"], "m": s["m"]}


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "quantize":
        x = s["x"].float()
        (v, e), (vt, et) = _quantize(x, case["block_rows"]), _quantize(x.t(), case["block_rows"])
        return {"x": _values(v, e, case["back"]), "xt": _values(vt, et, case["back"])}
    if op == "matmul":
        out = _decode(s["a"], s["sa"]) @ _decode(s["b"], s["sb"]).t()
        if s["bias"] is not None:
            out = out + s["bias"]
        return out.to(TYPES[case["out"]])
    if op == "muon":
        return _muon(s)
    ids = s["tokens"].long()
    here = (ids >= 0)[:, None]
    ids = ids.clamp_min(0)
    if op == "tokens_fwd":
        return torch.where(here, s["weight"][ids].float() * s["scale"], 0.0).to(TYPES[case["out"]])
    rows = torch.where(here, s["grad"].float() * s["scale"], 0.0)
    dw = torch.zeros(case["vocab"], case["dim"], device=rows.device).index_add_(0, ids, rows)
    return dw.to(TYPES[case["weight"]])


def run(state):
    if not own:
        return _plain(state)
    import sparse_ctr_embedding_gb300 as E

    s, case = state, state["case"]
    op = case["op"]
    if op == "quantize":
        q, e, qt, et = E.emb_fp4_quantize(s["x"], block_rows=case["block_rows"], transpose=True)
        rows, cols = s["x"].shape
        return {"x": E.emb_fp4_dequantize(q, e, cols, dtype=TYPES[case["back"]]),
                "xt": E.emb_fp4_dequantize(qt, et, rows, dtype=TYPES[case["back"]])}
    if op == "matmul":
        return E.emb_fp4_matmul(s["a"], s["sa"], s["b"], s["sb"], out_dtype=TYPES[case["out"]], bias=s["bias"],
                                workspace=s["workspace"])
    if op == "muon":
        s["opt"].step(s["grad"])
        return {"p": s["p"], "m": s["m"]}
    if op == "tokens_fwd":
        return E.emb_token_fwd(s["weight"], s["tokens"], scale=s["scale"], out_dtype=TYPES[case["out"]])
    return E.emb_token_bwd(s["grad"], s["tokens"], case["vocab"], scale=s["scale"], dtype=TYPES[case["weight"]],
                           workspace=s["workspace"])


# ------------------------------------------------------------------ 64 bits, from the definitions

def _exact_back(x, block_rows):
    """x rounded to the nearest of the block's 15 values, by their distance."""
    r, c = x.shape
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    out = torch.empty(r, c, dtype=torch.float64, device=x.device)
    step = max(block_rows, (1 << 26) // max(c, 1) // block_rows * block_rows)
    for at in range(0, r, step):
        t = x[at:at + step].double()
        n = t.shape[0]
        full = torch.nn.functional.pad(t, (0, -c % BLOCK, 0, -n % block_rows))
        top = full.abs().unflatten(1, (-1, BLOCK)).unflatten(0, (-1, block_rows)).amax((1, 3))
        unit = 2.0 ** torch.floor(torch.log2(top.clamp_min(2.0 ** -149)))
        unit = torch.where(unit > top, unit / 2, torch.where(2 * unit <= top, 2 * unit, unit))   # where the logarithm was rounded
        unit = (unit / 4).clamp(2.0 ** -127, 2.0 ** 125)
        unit = unit.repeat_interleave(block_rows, 0).repeat_interleave(BLOCK, 1)[:n, :c]
        mag = (t.abs() / unit).clamp_max(6.0)
        low = torch.searchsorted(grid, mag, right=True) - 1         # the grid value at or below, and the one above
        high = (low + 1).clamp_max(7)
        down, up = mag - grid[low], grid[high] - mag
        pick = torch.where((up < down) | ((up == down) & (high % 2 == 0)), high, low)
        out[at:at + step] = torch.sign(t) * grid[pick] * unit
    return out


def _exact_matrix(q, s, rows):
    """Rows of a quantised matrix in 64 bits, nibble by nibble."""
    part = q[rows].to(torch.int64)
    code = torch.empty(part.shape[0], 2 * part.shape[1], dtype=torch.int64, device=q.device)
    code[:, 0::2], code[:, 1::2] = part % 16, part // 16
    mag, sign = code % 8, 1.0 - 2.0 * (code // 8)
    frac, ex = mag % 2, mag // 2
    value = torch.where(ex == 0, 0.5 * frac, (1.0 + 0.5 * frac) * 2.0 ** (ex - 1.0))
    row = torch.arange(rows.start, rows.stop, device=q.device)[:, None]
    blk = torch.arange(code.shape[1], device=q.device)[None, :] // BLOCK
    e = s[row // 128, blk // 4, row % 32, row % 128 // 32, blk % 4]
    return sign * value * 2.0 ** (e.double() - 127.0)


def _exact_muon(s):
    a, b, c = NS
    beta, ps, ms = s["momentum"], [], []
    for p, g, m in zip(s["p"], s["grad"], s["m"]):
        g = g.double()
        m = m.double() + (1 - beta) * (g - m.double())
        u = g + beta * (m - g)
        u = u / (torch.linalg.norm(u) + 1e-7)
        # the same polynomial from the other side: X (a I + b X^T X + c (X^T X)^2), on the shorter side
        u = u if u.shape[0] >= u.shape[1] else u.t()
        for _ in range(NS_STEPS):
            z = u.t() @ u
            u = u @ (a * torch.eye(z.shape[0], dtype=z.dtype, device=z.device) + b * z + c * z @ z)
        u = u if u.shape == p.shape else u.t()
        ps.append(p.double() - s["lr"] * (s["weight_decay"] * p.double() + 0.2 * max(p.shape) ** 0.5 * u))
        ms.append(m)
    return {"p": ps, "m": ms}


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    op = case["op"]
    if op == "quantize":
        return {"x": _exact_back(s["x"], case["block_rows"]), "xt": _exact_back(s["x"].t(), case["block_rows"])}
    if op == "matmul":
        out = torch.empty(case["m"], case["n"], dtype=torch.float64, device="cuda")
        b = _exact_matrix(s["b"], s["sb"], slice(0, case["n"]))
        for r in range(0, case["m"], 16384):
            rows = slice(r, min(case["m"], r + 16384))
            out[rows] = _exact_matrix(s["a"], s["sa"], rows) @ b.t()
        return out if s["bias"] is None else out + s["bias"].double()
    if op == "muon":
        return _exact_muon(s)
    ids = s["tokens"].long()
    keep = torch.nonzero(ids >= 0)[:, 0]
    if op == "tokens_fwd":
        out = torch.zeros(case["n"], case["dim"], dtype=torch.float64, device="cuda")
        out[keep] = s["weight"].double().mul(s["scale"])[ids[keep]]
        return out
    out = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
    return out.index_put_((ids[keep],), s["grad"][keep].double(), accumulate=True) * s["scale"]
