"""From an encoder's last block to the loss and back, through the library's
calls alone: dropout of the block's output, the residual's addition and RMS
norm, a dense softmax head over the frequent labels and the group-shared sparse
layer over the tail; then scoring with the head kept in 8 bits.

    python examples/softmax_head.py [--rows 256] [--features 256] [--head 4096] [--steps 20]

The data is synthetic: each sample's features hold a noisy code of its head
label, so that the loss falls within a few steps.
"""
from __future__ import annotations

import argparse
import sys
from pathlib import Path

ROOT = Path(__file__).resolve().parents[1]
if str(ROOT) not in sys.path:
    sys.path.insert(0, str(ROOT))

import torch  # noqa: E402

import extreme_label_sparse_gb300 as sg  # noqa: E402

EPS, DROP, SMOOTHING, IGNORE = 1e-6, 0.1, 0.05, -100
GROUP, FAN_IN = 32, 64  # of the tail's groups


class Model:
    """Weights and buffers of one block's end, a dense head and a sparse tail."""

    def __init__(self, rows: int, features: int, head: int, tail: int, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        bf, f32, dev = torch.bfloat16, torch.float32, "cuda"

        def normal(*shape, std=1.0):
            return (torch.randn(shape, generator=g, device=dev) * std).to(bf)

        self.T, self.H, self.V, self.L = rows, features, head, tail
        self.weight = torch.ones(features, dtype=bf, device=dev)
        self.W = normal(head, features, std=features ** -0.5)
        groups = (torch.randperm(tail, generator=g, device=dev) // GROUP).to(torch.int32)
        idx = torch.stack([torch.randperm(features, generator=g, device=dev)[:FAN_IN] for _ in range(tail // GROUP)])
        self.layout = sg.sg_layout_build(groups, tail, GROUP, idx.to(torch.int32).reshape(-1), FAN_IN, features, rows,
                                         4 * rows)
        self.W_tail = normal(tail, FAN_IN, std=FAN_IN ** -0.5)
        # activations and gradients
        self.u, self.h, self.dh, self.du, self.dx = (torch.empty((rows, features), dtype=bf, device=dev)
                                                     for _ in range(5))
        self.rstd, self.loss, self.lse = (torch.empty(rows, dtype=f32, device=dev) for _ in range(3))
        self.dW, self.dW_tail = torch.empty_like(self.W), torch.empty_like(self.W_tail)
        self.dh_tail = torch.empty((rows, features), dtype=f32, device=dev)
        self.dweight = torch.empty(features, dtype=f32, device=dev)
        self.loss_tail = torch.zeros(1, dtype=torch.float64, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def step(self, x, residual, targets, rowptr, labels, seed: int, number: int, lr: float):
        """One training step; returns the mean losses of head and tail."""
        drop = dict(drop_p=DROP, seed=seed, offset=number)
        sg.sg_add_rmsnorm_fwd(x, self.weight, EPS, residual=residual, u=self.u, rstd=self.rstd, y=self.h, **drop)
        ce = dict(ignore_index=IGNORE, smoothing=SMOOTHING, status=self.status)
        sg.sg_softmax_ce_fwd(self.h, self.W, targets, self.loss, self.lse, **ce)
        dloss = torch.full((self.T,), 1.0 / self.T, device="cuda")
        sg.sg_softmax_ce_bwd(self.h, self.W, targets, self.lse, dloss, self.dh, self.dW, **ce)
        sg.sg_step(self.layout, self.h, self.W_tail, rowptr, labels, labels.numel(), self.dW_tail, self.dh_tail,
                   self.loss_tail)
        # both heads' gradients of h, then back through the norm and the dropout
        dh = (self.dh.float() + self.dh_tail / self.T).to(torch.bfloat16)
        sg.sg_add_rmsnorm_bwd(dh, self.u, self.weight, self.rstd, self.du, self.dweight, dx=self.dx, **drop)
        # a row's own label moves by about lr |h|^2 = lr H
        self.W.sub_(lr * self.T * self.dW)
        self.W_tail.sub_(lr / self.T * self.dW_tail)
        self.weight.sub_((0.01 * lr * self.dweight).to(torch.bfloat16))
        return self.loss.mean(), self.loss_tail / self.T

    def score(self, x, residual, targets):
        """Losses of rows against the head in 8 bits, as a server keeps it."""
        rows = x.shape[0]
        h8 = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
        hs, loss, lse = (torch.empty(rows, device="cuda") for _ in range(3))
        sg.sg_add_rmsnorm_fwd(x, self.weight, EPS, residual=residual, y8=h8, y8_scale=hs)
        top = self.W.float().abs().amax(1)
        W8, Ws = (self.W.float() * (448.0 / top)[:, None]).to(h8.dtype), top / 448.0
        sg.sg_softmax_ce_fwd(h8, W8, targets, loss, lse, h_scale=hs, W_scale=Ws, ignore_index=IGNORE,
                             status=self.status)
        return loss


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--rows", type=int, default=256)
    p.add_argument("--features", type=int, default=256)
    p.add_argument("--head", type=int, default=4096)
    p.add_argument("--tail", type=int, default=16384)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--lr", type=float, default=0.02)
    a = p.parse_args(argv)
    sg.build()
    m = Model(a.rows, a.features, a.head, a.tail)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    code = torch.randn((a.head, a.features), generator=g, device="cuda")
    rowptr = torch.arange(0, 3 * a.rows + 1, 3, dtype=torch.int32, device="cuda")
    history = []
    y = torch.randint(0, a.head, (a.rows,), generator=g, device="cuda", dtype=torch.int32)
    labels = torch.randint(0, a.tail, (3 * a.rows,), generator=g, device="cuda", dtype=torch.int32)
    residual = code[y.long()].to(torch.bfloat16)
    for i in range(a.steps):
        x = torch.randn((a.rows, a.features), generator=g, device="cuda").to(torch.bfloat16)
        sg.sg_dropout(x, DROP, 17, i, x)
        head, tail = m.step(x, residual, y, rowptr, labels, 23, i, a.lr)
        history.append((float(head), float(tail)))
        if i % 5 == 0 or i + 1 == a.steps:
            print(f"step {i}: softmax head {history[-1][0]:.4f}, sparse tail {history[-1][1]:.4f}")
    x = torch.zeros((8, a.features), dtype=torch.bfloat16, device="cuda")
    scored = m.score(x, residual[:8], y[:8])
    print("8-bit scores of 8 rows:", " ".join(f"{v:.3f}" for v in scored.tolist()))
    if int(m.status) or sg.sg_layout_status(m.layout):
        raise RuntimeError("a kernel reported " + sg.status_string(int(m.status) or sg.sg_layout_status(m.layout)))
    m.layout.close()
    return history, scored


if __name__ == "__main__":
    main()
