"""The end of an encoder's block and the next linear layer on 8-bit integers:
the norms around the block with its gate and residual scale, the layer's forward
pass on 8-bit rows, and both gradients from what was kept in 8 bits; then one
token at a time, as a server runs it.

    python examples/block8.py [--rows 256] [--features 512] [--outputs 1024] [--steps 20]

The data is synthetic: the targets are a fixed linear function of the normed rows.
"""
from __future__ import annotations

import argparse
import copy
import sys
from pathlib import Path

ROOT = Path(__file__).resolve().parents[1]
if str(ROOT) not in sys.path:
    sys.path.insert(0, str(ROOT))

import torch  # noqa: E402

import extreme_label_sparse_gb300 as sg  # noqa: E402

EPS = 1e-6


class Block:
    """Weights, and what a step keeps: x and u in 8 bits with a scale for 128
    columns, y in 8 bits with a scale for a row."""

    def __init__(self, rows: int, features: int, outputs: int, alpha: float = 1.0, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.alpha = alpha

        def new(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device="cuda")

        f32, i8, n = torch.float32, torch.int8, -(-features // 128)
        self.W = (torch.randn((outputs, features), generator=g, device="cuda") * features ** -0.5).bfloat16()
        self.post, self.gate, self.pre = (torch.ones(features, dtype=torch.bfloat16, device="cuda") for _ in range(3))
        self.W8, self.W_scale = new(outputs, features, dtype=i8), new(outputs, dtype=f32)
        self.u, self.dy, self.dx, self.dres = (new(rows, features) for _ in range(4))
        self.x8, self.u8, self.y8 = (new(rows, features, dtype=i8) for _ in range(3))
        self.x_scale, self.u_scale = new(rows, n, dtype=f32), new(rows, n, dtype=f32)
        self.rstd_x, self.rstd_u, self.y_scale = (new(rows, dtype=f32) for _ in range(3))
        self.z, self.dW = new(rows, outputs), new(outputs, features)
        self.dpost, self.dgate, self.dpre = (new(features, dtype=f32) for _ in range(3))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.pack()

    def first(self, rows: int):
        """This block, its weights among it, over its buffers' first rows."""
        b = copy.copy(self)
        for k in ("u", "dy", "dx", "dres", "x8", "u8", "y8", "x_scale", "u_scale", "rstd_x", "rstd_u", "y_scale", "z"):
            setattr(b, k, getattr(self, k)[:rows])
        return b

    def pack(self):
        """The layer's weights in 8 bits, a scale for each output."""
        sg.sg_pack8(self.W, self.W8, self.W_scale)

    def forward(self, x, residual):
        sg.sg_block_norm_fwd(x, self.post, self.pre, EPS, residual=residual, gate=self.gate, residual_scale=self.alpha,
                             u=self.u, rstd_x=self.rstd_x, rstd_u=self.rstd_u, y8=self.y8, y8_scale=self.y_scale,
                             x8=self.x8, x_scale=self.x_scale, u8=self.u8, u_scale=self.u_scale)
        sg.sg_linear8_fwd(self.y8, self.y_scale, self.W8, self.W_scale, self.z, status=self.status)
        return self.z

    def backward(self, dz, du_in=None):
        """From dz and the gradient that reaches u by the residual, to those of x,
        the residual and the weights.  x and u are not needed any more."""
        sg.sg_linear8_bwd(self.y8, self.y_scale, self.W8, self.W_scale, dz, dx=self.dy, dW=self.dW, status=self.status)
        sg.sg_block_norm_bwd(self.dy, self.u8, self.x8, self.post, self.pre, self.rstd_x, self.rstd_u, self.dx,
                             dresidual=self.dres, dpost=self.dpost, dpre=self.dpre, dgate=self.dgate, gate=self.gate,
                             residual_scale=self.alpha, du_in=du_in, u_scale=self.u_scale, x_scale=self.x_scale)

    def update(self, lr: float):
        self.W.sub_(lr * self.dW)
        for w, d in ((self.post, self.dpost), (self.gate, self.dgate), (self.pre, self.dpre)):
            w.sub_((0.01 * lr * d).bfloat16())
        self.pack()


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--rows", type=int, default=256)
    p.add_argument("--features", type=int, default=512)
    p.add_argument("--outputs", type=int, default=1024)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--lr", type=float, default=0.2)
    a = p.parse_args(argv)
    sg.build()
    b = Block(a.rows, a.features, a.outputs)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, res = (torch.randn((a.rows, a.features), generator=g, device="cuda").bfloat16() for _ in range(2))
    want = torch.randn((a.rows, a.outputs), generator=g, device="cuda")
    # the largest curvature of the mean square over the rows is about twice this
    lr = a.lr / (1 + (a.features / a.rows) ** 0.5) ** 2
    losses = []
    for i in range(a.steps):
        z = b.forward(x, res)
        diff = z.float() - want
        losses.append(float(diff.square().mean()))
        b.backward((diff * (2.0 / a.rows)).bfloat16())
        b.update(lr)
        if i % 5 == 0 or i + 1 == a.steps:
            print(f"step {i}: mean square error {losses[-1]:.4f}")
    # one token at a time, in the same buffers' first rows
    one = b.first(1)
    served = torch.cat([one.forward(x[i:i + 1], res[i:i + 1]).clone() for i in range(min(4, a.rows))])
    if int(b.status):
        raise RuntimeError("a kernel reported " + sg.status_string(int(b.status)))
    print("served", tuple(served.shape), "largest", float(served.abs().max()))
    return b, losses, served


if __name__ == "__main__":
    main()
