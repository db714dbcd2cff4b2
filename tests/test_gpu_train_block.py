"""The residual block of examples/train_block.py: its loss falls, and its hand-written backward
pass agrees with differences of its loss along each parameter's gradient."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _block(n_nodes, p):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    try:
        from train_block import Block
    finally:
        sys.path.pop(0)
    return Block(n_nodes, p)


def test_loss_falls():
    losses = _block(300, 0.1).train(30)
    print(f"[gpu-test] losses {losses[0]:.4f} -> {losses[-1]:.4f}", flush=True)
    assert all(v == v for v in losses) and losses[-1] < 0.5 * losses[0]


def test_gradients_against_differences():
    """With one set of masks the loss is a smooth function of each parameter.  Central
    differences with a step of 1e-2 along the gradient's unit direction: the loss, of order
    one to ten, carries about 1e-6 of itself in fp32 rounding, so the quotient about 1e-3 at
    the most; the third-order term, 1e-4 / 6 of the third derivative, is of that size too.
    Held to 1 % of the gradient's length plus 2e-3."""
    block = _block(300, 0.2)
    _, grads = block.step(3)
    for name, g in grads.items():
        d = g / g.norm()
        base = block.params[name].clone()
        loss = []
        for sign in (1, -1):
            block.params[name] = base + sign * 1e-2 * d
            loss.append(float(block.step(3)[0]))
        block.params[name] = base
        diff, want = (loss[0] - loss[1]) / 2e-2, float((g * d).sum())
        print(f"[gpu-test] d loss / d {name}: {want:.5f}, differences {diff:.5f}", flush=True)
        assert abs(diff - want) <= 1e-2 * abs(want) + 2e-3, name
