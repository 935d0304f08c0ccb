"""Plain forms of the 4-bit operators (test code only): the microscaling format's
encoding by its definition in 64 bits on the host, and the product's error bound.

A product's sums: products of two codes are exact; within one tensor-core step up
to 64 of them are added, each possibly cut at the width of the largest (2 u of the sum
of magnitudes per term, 128 u); then ceil(k/64) step sums, pieces of a split and the bias
are added one after the other (2 u each, since tensor cores may cut instead of round).
u = 2^-24 is the float32 rounding unit.
"""
from __future__ import annotations

import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def encode(x, block_rows):
    """Codes uint8[rows, cols] and scale bytes uint8[rows, ceil(cols/32)] of a matrix, by the definition."""
    x = x.double()
    r, c = x.shape
    full = torch.zeros(-(-r // block_rows) * block_rows, -(-c // 32) * 32, dtype=torch.float64)
    full[:r, :c] = x
    blocks = full.view(full.shape[0] // block_rows, block_rows, full.shape[1] // 32, 32)
    amax = blocks.abs().nan_to_num(nan=float("inf"), posinf=float("inf")).amax((1, 3))
    _, ex = torch.frexp(amax)                     # amax in [2^(ex-1), 2^ex)
    e = (ex - 1 - 2).clamp_min(-127)
    e = torch.where(amax == 0, -127, e)
    byte = torch.where(torch.isinf(amax), 255, e + 127)
    e_el = e.repeat_interleave(block_rows, 0).repeat_interleave(32, 1)[:r, :c]
    mag = torch.ldexp(x.abs(), -e_el)
    # nearest of the grid; a tie goes to the code with an even number
    dist = (mag.nan_to_num(0.0, 0.0).clamp_max(6.0)[..., None] - GRID).abs()
    best = dist.amin(-1, keepdim=True)
    hit = dist == best
    number = torch.arange(8)
    code = torch.where(hit & (number % 2 == 0), number, torch.where(hit, number + 100, 1000)).amin(-1) % 100
    code = code + 8 * torch.signbit(x)
    return code.to(torch.uint8), byte.repeat_interleave(block_rows, 0)[:r].to(torch.uint8)


def pack(code):
    r, c = code.shape
    p = torch.zeros(r, -(-c // 2) * 2, dtype=torch.uint8)
    p[:, :c] = code
    return p[:, 0::2] | (p[:, 1::2] << 4)


def unpack(q, cols):
    q = q.cpu()
    return torch.stack([q & 15, q >> 4], 2).view(q.shape[0], -1)[:, :cols]


def untile(s, rows, blocks):
    """Scale bytes [rows, blocks] from the tiled order, element by element of its definition."""
    r, b = torch.arange(rows)[:, None], torch.arange(blocks)[None, :]
    return s.cpu()[r // 128, b // 4, r % 32, r % 128 // 32, b % 4]


def tile(e):
    r, b = e.shape
    s = torch.zeros(-(-r // 128), -(-b // 4), 32, 4, 4, dtype=torch.uint8)
    ri, bi = torch.arange(r)[:, None], torch.arange(b)[None, :]
    s[ri // 128, bi // 4, ri % 32, ri % 128 // 32, bi % 4] = e
    return s


def values(code, byte):
    """The 64-bit matrix that codes and scale bytes stand for (255: NaN)."""
    c = code.long()
    v = GRID[c % 8] * (1 - 2 * (c // 8))
    e = byte.repeat_interleave(32, 1)[:, :code.shape[1]].double() - 127
    return torch.where(e == 128, float("nan"), v * 2.0 ** e)


def ulps(k, pieces=152):
    """pieces: of a tile, at most one a step and one an SM."""
    return 128 + 2 * (-(-k // 64)) + 2 * min(-(-k // 256), pieces) + 4
