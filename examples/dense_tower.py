"""One CTR training step end to end: pooled embeddings, a dense tower, both optimizers.

The sparse half is the library's embedding step (emb_lookup_fwd_record,
emb_bwd_adagrad_recorded).  On its pooled output [B, sum_dims] runs a tower of
gated residual blocks, every layer through the dense operators:

  x    = pooled W_in^T + b_in                          8-bit product
  h    = norm(x) w_pre[0]                              first norm
  f, g = h W_f^T, h W_g^T                              8-bit products, per block
  x    = x + sigmoid(g) (norm(f) w_post);  h = norm(x) w_pre[i+1]
  p    = sigmoid(h w_out)

Each activation and gradient is quantised once, along its rows for the products
that contract its features and along the batch for the weight gradients; each
weight once a step, in 128 x 128 blocks.  The weights are trained by AdamW with
8-bit states, the embeddings by sparse Adagrad.

  python examples/dense_tower.py [steps]
"""
from __future__ import annotations

import os
import sys
from typing import List

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_ctr_embedding_gb300 as E  # noqa: E402
import workload as W  # noqa: E402


class Tower:
    """The dense weights, their forward and their backward."""

    def __init__(self, in_dim: int, width: int, blocks: int, seed: int = 0, state: str = "q8", lr: float = 3e-3):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(o, i):
            return torch.randn(o, i, device="cuda", generator=g) * i ** -0.5

        self.blocks = blocks
        self.p = {"w_in": weight(width, in_dim), "b_in": torch.zeros(width, device="cuda"),
                  "w_out": torch.zeros(width, device="cuda")}
        for i in range(blocks):
            self.p.update({f"w_f{i}": weight(width, width), f"w_g{i}": weight(width, width),
                           f"post{i}": torch.ones(width, device="cuda"), f"pre{i}": torch.ones(width, device="cuda")})
        self.p[f"pre{blocks}"] = torch.ones(width, device="cuda")
        self.names = list(self.p)
        self.opt = E.AdamW([self.p[k] for k in self.names], lr=lr, state=state, seed=seed)

    def forward(self, pooled: torch.Tensor) -> torch.Tensor:
        """Logits [B]; keeps what the backward needs."""
        p, k = self.p, {}
        k["in"] = E.emb_fp8_quantize(pooled, 1, transpose=True)
        for name in self.names:
            if p[name].dim() == 2:
                k[name] = E.emb_fp8_quantize(p[name], 128, transpose=True)
        x = E.emb_fp8_matmul(*k["in"][:2], *k["w_in"][:2], out_dtype=torch.float32, bias=p["b_in"])
        _, h, stats = E.emb_norm_gate_fwd(x, None, w_pre=p["pre0"], block_dtype=torch.bfloat16)
        k["x"], k["first"] = x, stats
        for i in range(self.blocks):
            q = k[f"h{i}"] = E.emb_fp8_quantize(h, 1, transpose=True)
            f, gate = (E.emb_fp8_matmul(*q[:2], *k[f"{w}{i}"][:2]) for w in ("w_f", "w_g"))
            x, h, stats = E.emb_norm_gate_fwd(x, f, gate, w_post=p[f"post{i}"], w_pre=p[f"pre{i + 1}"])
            k[f"y{i}"] = (x, f, gate, stats)
        k["h"], self.kept = h, k
        return h.float() @ p["w_out"]

    def backward(self, dlogits: torch.Tensor) -> torch.Tensor:
        """Steps the dense weights; returns the gradient of the pooled embeddings."""
        p, k, grad = self.p, self.kept, {}
        grad["w_out"] = dlogits @ k["h"].float()
        dh = (dlogits[:, None] * p["w_out"]).to(torch.bfloat16)
        dx = None
        for i in reversed(range(self.blocks)):
            y, f, gate, stats = k[f"y{i}"]
            d = E.emb_norm_gate_bwd(dx, dh, y, f, gate, stats, w_post=p[f"post{i}"], w_pre=p[f"pre{i + 1}"])
            dx, grad[f"post{i}"], grad[f"pre{i + 1}"] = d["dx"], d["dw_post"], d["dw_pre"]
            dh = 0
            for w, part in (("w_f", d["df"]), ("w_g", d["dgate"])):
                q, s, qt, st = E.emb_fp8_quantize(part, 1, transpose=True)
                grad[f"{w}{i}"] = E.emb_fp8_matmul(qt, st, *k[f"h{i}"][2:], out_dtype=torch.float32)
                dh = dh + E.emb_fp8_matmul(q, s, *k[f"{w}{i}"][2:], out_dtype=torch.float32)
            dh = dh.to(torch.bfloat16)
        d = E.emb_norm_gate_bwd(dx, dh, k["x"], None, None, k["first"], w_pre=p["pre0"])
        grad["pre0"], dx = d["dw_pre"], d["dx"]
        q, s, qt, st = E.emb_fp8_quantize(dx, 1, transpose=True)
        grad["b_in"] = dx.sum(0)
        grad["w_in"] = E.emb_fp8_matmul(qt, st, *k["in"][2:], out_dtype=torch.float32)
        dpooled = E.emb_fp8_matmul(q, s, *k["w_in"][2:], out_dtype=torch.float32)
        self.opt.step([grad[n] for n in self.names])
        return dpooled


def train(steps: int = 60, cfg=None, width: int = 192, blocks: int = 2, state: str = "q8") -> List[float]:
    """Fits the labels of one synthetic batch; returns the loss of every step."""
    cfg = cfg or W.config(1)
    wl = W.make(cfg, device="cuda")
    table = E.emb_table_create(cfg.dims, cfg.wdtype, wl.keys.cpu(), values=wl.values, capacity=cfg.capacity, acc_init=cfg.acc0)
    ws = torch.empty(E.emb_bwd_workspace_size(table, cfg.n_bags, wl.qkeys.numel()), dtype=torch.uint8, device="cuda")
    tower = Tower(cfg.sum_dims, width, blocks, state=state)
    labels = (torch.rand(cfg.batch, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) < 0.3).float()
    losses = []
    for _ in range(steps):
        pooled = E.emb_lookup_fwd_record(table, wl.offsets, wl.qkeys, cfg.pool, ws)
        logits = tower.forward(pooled)
        losses.append(torch.nn.functional.binary_cross_entropy_with_logits(logits, labels))
        dpooled = tower.backward((torch.sigmoid(logits) - labels) / cfg.batch)
        E.emb_bwd_adagrad_recorded(table, cfg.n_bags, wl.qkeys.numel(), cfg.pool, dpooled, cfg.lr, cfg.eps, ws)
    if E.emb_check_device_flag(table) or E.emb_check_op_flag():
        raise RuntimeError("a kernel reported bad input or gave up a wait")
    table.close()
    return [float(v) for v in losses]


if __name__ == "__main__":
    out = train(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
    for i in range(0, len(out), max(1, len(out) // 10)):
        print(f"step {i}: loss {out[i]:.4f}")
    print(f"step {len(out) - 1}: loss {out[-1]:.4f}")
