"""The feed-forward block of examples/train_feedforward.py: it runs, and its hand-written backward pass agrees
with float64 automatic differentiation of the same formulas on the CPU.

Tolerance: the longest chain is two products, two norms and a product again, each within about
1e-5 of its terms' magnitudes in fp32 (sums of up to 300 rows and 128 columns); held to 1e-4 of a
gradient's largest number."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _block(n_nodes):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    try:
        from train_feedforward import FeedForward
    finally:
        sys.path.pop(0)
    return FeedForward(n_nodes)


def _norm(x, w, b):
    var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    return (x - mean) / torch.sqrt(var + 1e-5) * w + b


def test_gradients():
    block = _block(300)
    loss, grads = block.step()
    q = {k: v.double().cpu().requires_grad_() for k, v in block.params.items()}
    s = block.s.double().cpu()
    u = torch.nn.functional.silu(s @ q["A"] + q["a"])
    h = s + q["scale"] * torch.sigmoid(s @ q["G"] + q["d"]) * _norm(u @ q["B"] + q["b"], q["w1"], q["b1"])
    want = ((_norm(h, q["w2"], q["b2"]) @ q["c"] - block.target.double().cpu()) ** 2).mean()
    want.backward()
    assert abs(float(loss) - float(want.detach())) <= 1e-4 * abs(float(want.detach()))
    for name, g in grads.items():
        ref = q[name].grad
        d = float((g.double().cpu() - ref).abs().max() / ref.abs().max())
        print(f"[gpu-test] gradient of {name}: {d:.2e}", flush=True)
        assert g.shape == ref.shape and d <= 1e-4, name


def test_runs():
    log = _block(300).train(5)
    assert len(log) == 5 and all(v == v and v < float("inf") for pair in log for v in pair)
