"""Plain 64-bit forms of the dense-tower operators, and the error bounds their
kernels are held to (test code only).

u = 2^-24 is the float32 rounding unit.  Bounds are set from the arithmetic,
before any run: a float32 result may differ from the 64-bit one by a small
multiple of u times the sum of the magnitudes of what was added to form it
(the `size` arrays below), plus one rounding to the output's own type.

* A row sum of up to 8192 terms takes 8 sequential and 10 pairwise additions:
  18 u relative to the sum of magnitudes.  A norm adds a division, a square
  root and four products, a gate an exponential and a division (4 u): 40 u in
  all for the forward.  The backward chains two such norms: 128 u.
* Sums over R rows add at most R sequential roundings: (R + 128) u.
* A matrix product of k terms adds them in blocks of 128 (each block in any
  order, at most 2 u an addition since tensor cores may cut instead of round:
  256 u) and ceil(k/128) block sums with a scale each: (256 + ceil(k/128) + 4) u.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # float32: within the u terms
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}


def close(name, x, ref, size, ulps):
    """|x - ref| <= ulps u size + one rounding of x's type, element by element."""
    x64, ref = x.detach().cpu().double(), ref.cpu()
    tol = ulps * U * size.cpu() + ROUND[x.dtype] * ref.abs() + TINY[x.dtype]
    bad = ~((x64 - ref).abs() <= tol)
    if bad.any():
        i = int(bad.flatten().nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())}/{bad.numel()} outside; at {i}: {x64.flatten()[i].item()} "
                             f"against {ref.flatten()[i].item()}, bound {tol.flatten()[i].item()}")


def act64(gate, act):
    if gate is None:
        return torch.ones((), dtype=torch.float64)
    return 1 / (1 + torch.exp(-gate)) if act == "sigmoid" else gate


def norm64(t, w, b, layer, eps):
    if layer:
        t = t - t.mean(1, keepdim=True)
    t = t / torch.sqrt((t * t).mean(1, keepdim=True) + eps)
    t = t if w is None else t * w
    return t if b is None else t + b


def norm_size(t, w, b, layer, eps):
    """Magnitude of the terms behind each element of norm64."""
    c = t - t.mean(1, keepdim=True) if layer else t
    big = t.abs() + (t.abs().mean(1, keepdim=True) if layer else 0)
    s = big / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    # an error of the mean also changes the variance: relative to sigma, by (mean |t| / sigma) of itself
    s = s * (big.mean(1, keepdim=True) / torch.sqrt((c * c).mean(1, keepdim=True) + eps)).clamp_min(1.0)
    s = s if w is None else s * w.abs()
    return s if b is None else s + b.abs()


def block_scales(x, block_rows):
    """Quantiser in float32, as it is defined: codes (float8) and scales."""
    r, c = x.shape
    t = torch.nn.functional.pad(x.float(), (0, -c % 128, 0, -r % block_rows))
    t = t.reshape(t.shape[0] // block_rows, block_rows, t.shape[1] // 128, 128)
    mag = torch.where(t.abs() <= torch.finfo(torch.float32).max, t.abs(), torch.zeros_like(t))
    amax = mag.amax((1, 3), keepdim=True).clamp_min(1e-30)
    q = torch.where(t.abs() <= torch.finfo(torch.float32).max, t * (448.0 / amax), torch.full_like(t, float("nan")))
    s = (amax * (1.0 / 448.0))[:, 0, :, 0].t().contiguous()
    q = q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.reshape(t.shape[0] * block_rows, -1)[:r, :c], s


def dequant64(q, s):
    r, c = q.shape
    s = s.double()
    s = s if s.shape[1] == r else s.repeat_interleave(128, 1)[:, :r]
    return q.float().double() * s.t().repeat_interleave(128, 1)[:, :c]


def fmix32(h):
    low = 0xFFFFFFFF
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & low
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & low
    return h ^ (h >> 16)


def random_bits(first, n, seed, step):
    i = first + torch.arange(n, dtype=torch.int64)
    key = (seed * 0x9E3779B9 + step * 0x85EBCA6B) & 0xFFFFFFFF
    return fmix32((i & 0xFFFFFFFF) ^ (((i >> 32) * 0x9E3779B9) & 0xFFFFFFFF) ^ key)


def e4m3_values():
    """All non-negative finite codes' values, ascending (index = code)."""
    return torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()


def round_state(t, r16):
    """States to codes, by searching the code table: the value lies between two
    codes, and the upper one is taken when the 16 random bits (and a half) plus
    the value's place between them, in 2^-20 steps of its bits, reach 2^20."""
    n = t.numel()
    pad = torch.nn.functional.pad(t, (0, -n % 256)).view(-1, 256)
    finite = pad.abs() <= torch.finfo(torch.float32).max
    amax = torch.where(finite, pad.abs(), torch.zeros_like(pad)).amax(1, keepdim=True).clamp_min(1e-30)
    x = (pad * (448.0 / amax)).reshape(-1)[:n]
    scale = (amax * (1.0 / 448.0)).reshape(-1)
    vals = e4m3_values().double()
    mag = x.abs().clamp_max(448.0).double()
    ok = torch.isfinite(t)
    mag = torch.where(ok, mag, torch.zeros_like(mag))
    lo = torch.searchsorted(vals, mag, right=True) - 1
    hi = (lo + 1).clamp_max(126)
    gap = (vals[hi] - vals[lo]).clamp_min(1e-300)
    # below 2^-6 the value is first rounded to steps of 2^-29 (2^-20 of a gap)
    frac = torch.where(mag < 2.0 ** -6, torch.round(mag * 2.0 ** 29) * 2.0 ** -29 - vals[lo], mag - vals[lo]) / gap
    up = torch.floor(frac * 2 ** 20) + (r16 * 16 + 8).double() >= 2 ** 20
    code = torch.where(up, hi, lo)
    neg = (x < 0) & ok
    out = torch.where(neg, -vals[code], vals[code]).float()
    out = torch.where(ok, out, torch.full_like(out, float("nan")))
    return out, scale


def adamw32(p, g, m, v, u, hyper, q8, first=0, grad_scale=None):
    """One step in float32, each operation rounded by itself.  v for float32
    states, u (the dequantised root) for 8-bit ones.  Returns (p, m, v, u)."""
    lr, b1, b2, eps, wd, step = hyper
    g = g.float()
    if grad_scale is not None:
        g = g * torch.tensor(grad_scale, dtype=torch.float32)
    v = u * u if q8 else v
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    u = torch.sqrt(v)
    den = u * (1.0 / (1.0 - b2 ** step) ** 0.5) + eps
    w = p.float() * (1.0 - lr * wd) - (m * (lr / (1.0 - b1 ** step))) / den
    return w, m, v, u
