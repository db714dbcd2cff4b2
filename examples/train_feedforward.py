"""Train a gated feed-forward block on the invariants of a convolution, forward and backward by hand.

    python examples/train_feedforward.py [--nodes 600] [--steps 20]

On a radius graph, with s the 64 scalars of the convolution's output (a strided view), the block computes

    u = silu(s A + a)                                etpc_linear, 64 -> 128
    v = u B + b                                      etpc_linear, 128 -> 64
    g = s G + d                                      etpc_linear, the gate's logits
    h = s + scale sigmoid(g) norm(v), y = norm(h)    etpc_norm_gate_add_norm
    e = y c                                          etpc_linear, one number a node

and fits e to a number of each node by gradient descent, all gradients clipped to a global norm
(etpc_clip_grad_norm).
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

C, HIDDEN = 64, 128


class FeedForward:
    """The block's inputs, parameters and target on the GPU."""

    def __init__(self, n_nodes: int, seed: int = 11):
        cfg = small_variant("cfg5", n_nodes)
        plan = etpc.Plan(cfg.irreps_in, cfg.irreps_out, cfg.lmax_sh, cfg.mode, cfg.radial, cfg.n_basis, cfg.r_lo, cfg.r_hi,
                         cfg.poly_p, box=cfg.box)
        wl = make_workload(cfg, w_blocks=plan.w_blocks(), z_dim=plan.info()["z_dim"],
                           scalar_out_mask=np.ones(plan.info()["z_dim"], bool))
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        x, pos = dev(wl.x), dev(wl.pos)
        graph = etpc.etpc_csr_build(cfg.n_nodes, dev(wl.src), dev(wl.dst), pos=pos, box=cfg.box and (cfg.box,) * 3)
        self.features = etpc.etpc_forward(plan, graph, x, pos, dev(wl.w))
        self.s = self.features[:, :C]
        gen = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *n: torch.randn(*n, generator=gen, device="cuda")  # noqa: E731
        ones, zeros = (lambda n: torch.ones(n, device="cuda")), (lambda n: torch.zeros(n, device="cuda"))
        self.params = dict(A=normal(C, HIDDEN) / C ** 0.5, a=zeros(HIDDEN), B=normal(HIDDEN, C) / HIDDEN ** 0.5, b=zeros(C),
                           G=normal(C, C) / C ** 0.5, d=zeros(C), w1=ones(C), b1=zeros(C), scale=ones(C), w2=ones(C), b2=zeros(C),
                           c=normal(C, 1) / C ** 0.5)
        self.target = 3.0 * x[:, :C].mean(1, keepdim=True)

    def step(self):
        """(loss, gradients of the parameters)."""
        q, s, n = self.params, self.s, self.s.shape[0]
        u, zu = etpc.etpc_linear(s, q["A"], q["a"], act="silu")
        v, _ = etpc.etpc_linear(u, q["B"], q["b"])
        g, _ = etpc.etpc_linear(s, q["G"], q["d"])
        norms = dict(w1=q["w1"], b1=q["b1"], scale=q["scale"], w2=q["w2"])
        y, h, stats = etpc.etpc_norm_gate_add_norm(v, gate=g, residual=s, b2=q["b2"], **norms)
        e, _ = etpc.etpc_linear(y, q["c"])
        err = e - self.target
        loss = err.square().mean()

        grads = {}
        y_bar, grads["c"], _ = etpc.etpc_linear_backward(y, q["c"], (2.0 / n) * err, want=("x", "w"))
        v_bar, g_bar, _, grads["w1"], grads["b1"], grads["scale"], grads["w2"], grads["b2"] = \
            etpc.etpc_norm_gate_add_norm_backward(v, h, y_bar, stats, gate=g, **norms)
        _, grads["G"], grads["d"] = etpc.etpc_linear_backward(s, q["G"], g_bar, want=("w", "b"))
        u_bar, grads["B"], grads["b"] = etpc.etpc_linear_backward(u, q["B"], v_bar)
        _, grads["A"], grads["a"] = etpc.etpc_linear_backward(s, q["A"], u_bar, z=zu, act="silu", want=("w", "b"))
        return loss, grads

    def train(self, steps: int, rate: float = 0.05, max_norm: float = 1.0):
        """Gradient descent with clipped gradients; returns (loss, norm) of each step."""
        log = []
        for _ in range(steps):
            loss, grads = self.step()
            norm = etpc.etpc_clip_grad_norm(list(grads.values()), max_norm)
            log.append((float(loss), float(norm)))
            for name, g in grads.items():
                self.params[name] -= rate * g
        return log


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--nodes", type=int, default=600)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    for k, (loss, norm) in enumerate(FeedForward(a.nodes).train(a.steps)):
        print(f"step {k:3d}  loss {loss:.5f}  gradient norm {norm:.4f}", flush=True)


if __name__ == "__main__":
    main()
