"""Train one residual block around the convolution, forward and backward by hand.

    python examples/train_block.py [--nodes 600] [--steps 20]

On a radius graph with 64x0e+64x1o+64x2e features x, the block computes

    z = conv(x, pos, W)                              etpc_forward
    h = x + dropout(z)                               etpc_irreps_dropout (whole channels)
    v = irreps_norm(h)                               etpc_irreps_norm
    s = the 64 scalars of v, u = s A                 (a strided view; torch matrix product)
    y = layer_norm(s + dropout(u))                   etpc_dropout_add_layer_norm
    e = y c                                          one number a node

and fits e to the scalars' mean of x by gradient descent on W, A, c and the norms' gains
and biases.  Every backward call repeats the forward pass's (seed, offset); the offset is the
step, so each step has its own masks.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import equivariant_gnn_tensor_amd as etpc  # noqa: E402
from workloads import make_workload, small_variant  # noqa: E402

C = 64   # channels of every block


class Block:
    """The block's plan, graph, parameters and training data on the GPU."""

    def __init__(self, n_nodes: int, p: float, seed: int = 11):
        cfg = small_variant("cfg5", n_nodes)
        self.irreps, self.p, self.seed = cfg.irreps_in, p, seed
        self.plan = etpc.Plan(cfg.irreps_in, cfg.irreps_out, cfg.lmax_sh, cfg.mode, cfg.radial, cfg.n_basis, cfg.r_lo,
                              cfg.r_hi, cfg.poly_p, box=cfg.box)
        wl = make_workload(cfg, w_blocks=self.plan.w_blocks(), z_dim=self.plan.info()["z_dim"],
                           scalar_out_mask=np.ones(self.plan.info()["z_dim"], bool))
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.x, self.pos = dev(wl.x), dev(wl.pos)
        self.graph = etpc.etpc_csr_build(cfg.n_nodes, dev(wl.src), dev(wl.dst), pos=self.pos, box=cfg.box and (cfg.box,) * 3)
        dims = etpc.etpc_irreps_dims(self.irreps)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        ones, zeros = (lambda n: torch.ones(n, device="cuda")), (lambda n: torch.zeros(n, device="cuda"))
        self.params = dict(W=dev(wl.w), g=ones(dims["channels"]), b=zeros(dims["biases"]), A=normal(C, C) / C ** 0.5,
                           g2=ones(C), b2=zeros(C), c=normal(C) / C ** 0.5)
        self.target = 3.0 * self.x[:, :C].mean(1)

    def step(self, offset: int):
        """(loss, gradients of the parameters) with the masks of `offset`."""
        q, n = self.params, self.x.shape[0]
        drop = dict(p=self.p, seed=self.seed, offset=2 * offset)
        drop2 = dict(p=self.p, seed=self.seed, offset=2 * offset + 1)
        z = etpc.etpc_forward(self.plan, self.graph, self.x, self.pos, q["W"])
        h = self.x + etpc.etpc_irreps_dropout(self.irreps, z, **drop)
        v, stats = etpc.etpc_irreps_norm(self.irreps, h, q["g"], q["b"])
        s = v[:, :C]
        y, h2, mean, rstd = etpc.etpc_dropout_add_layer_norm(s @ q["A"], s, q["g2"], q["b2"], **drop2)
        err = y @ q["c"] - self.target
        loss = err.square().mean()

        e_bar = (2.0 / n) * err
        grads = dict(c=y.t() @ e_bar)
        y_bar = e_bar[:, None] * q["c"]
        u_bar, s_bar, grads["g2"], grads["b2"] = etpc.etpc_dropout_add_layer_norm_backward(h2, y_bar, mean, rstd, q["g2"],
                                                                                           **drop2)
        grads["A"] = s.t() @ u_bar
        v_bar = torch.zeros_like(v)
        v_bar[:, :C] = s_bar + u_bar @ q["A"].t()
        h_bar, grads["g"], grads["b"] = etpc.etpc_irreps_norm_backward(self.irreps, h, v_bar, stats, q["g"])
        z_bar = etpc.etpc_irreps_dropout(self.irreps, h_bar, **drop)
        _, grads["W"], _ = etpc.etpc_backward(self.plan, self.graph, self.x, self.pos, q["W"], z_bar, want=("w",))
        return loss, grads

    def train(self, steps: int, rate: float = 0.05):
        """Plain gradient descent; returns the losses."""
        losses = []
        for k in range(steps):
            loss, grads = self.step(k)
            losses.append(float(loss))
            for name, g in grads.items():
                self.params[name] -= rate * g
        return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--nodes", type=int, default=600)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--dropout", type=float, default=0.1)
    a = ap.parse_args()
    for k, loss in enumerate(Block(a.nodes, a.dropout).train(a.steps)):
        print(f"step {k:3d}  loss {loss:.5f}", flush=True)


if __name__ == "__main__":
    main()
