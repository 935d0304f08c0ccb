"""Muon by its definition in 64 bits, and a form of it that rounds where the kernels
round (test code only).

The form with `planes` keeps X, A and B as float16 (times 2^12), one or two of each, and
everything else in 64 bits.  Its distance from the exact form is what one rounding
to float16 of every value costs, the steps' own magnification included; the kernels
make the same roundings, of values that differ by their float32 sums' 2^-24 or so.  That
is not the same result: a value near a border rounds to its other neighbour, and from
there on all later values, hence their roundings, are other ones (float32 on the host
against the 64-bit form: 64 x 64, seed 65 of the tests' data, no value differs in the first
step, 3 of 100 in the third, 87 of 100 in the fifth, and the ends are 0.56 of that distance
apart).  So a kernel's error is another draw of errors of the same size, not the same errors:
it is held to 3 times the distance from the exact form, plus 64 u of the update for
the float32 around it (u = 2^-24).
"""
from __future__ import annotations

import torch

A, B, C = 3.4445, -4.7750, 2.0315
S = 4096.0


def momentum(g, m, beta, nesterov=True):
    g, m = g.double(), m.double()
    m = beta * m + (1 - beta) * g
    return m, ((1 - beta) * g + beta * m if nesterov else m)


def _planes(x, planes):
    hi = (x * S).to(torch.float16).double()
    if planes == 1:
        return hi / S, torch.zeros_like(x)
    return hi / S, (x * S - hi).to(torch.float16).double() / S


def _product(x, y):
    return x[0] @ y[0] + x[0] @ y[1] + x[1] @ y[0]


def orthogonal(u, planes=None):
    """Five steps on u / (|u| + 1e-7) in 64 bits (planes None), or with float16 matrices."""
    keep = (lambda t: (t, torch.zeros_like(t))) if planes is None else (lambda t: _planes(t, planes))
    x = u / (u.norm() + 1e-7)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t()
    for _ in range(5):
        px = keep(x)
        pa = keep(_product(px, (px[0].t(), px[1].t())))
        pb = keep(B * (pa[0] + pa[1]) + C * _product(pa, pa))
        x = A * (px[0] + px[1]) + _product(pb, px)
    return x.t() if tall else x
