"""GPU checks of the gradient norm and clipping against oracle/feedforward.py (float64).

Squares and sums are taken in 64 bits (far below the tolerances), so the norm is off by its rounding to
fp32, and a clipped gradient by the rounding of the factor to fp32, of the product (both 2^-24) and of
the result to its type (half a step).
"""
import math

import numpy as np
import pytest
import torch

from oracle import feedforward as ff
from tests.gpu_helpers import note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LEAST = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _etpc():
    import equivariant_gnn_tensor_amd as etpc
    return etpc


def f64(t):
    return t.detach().double().cpu().numpy()


def tensors(rng, sizes, kinds, scale=0.1, shift=0):
    """Tensors that start `shift` elements into their buffers."""
    out = []
    for k, n in enumerate(sizes):
        full = torch.zeros(n + shift, dtype=DTYPES[kinds[k % len(kinds)]], device="cuda")
        full[shift:] = torch.from_numpy(scale * rng.standard_normal(n)).to("cuda", full.dtype)
        out.append(full[shift:])
    return out


def check_norm(got, ref):
    assert got.dtype == torch.float32 and abs(float(got) - ref) <= 2 * U * ref, (float(got), ref)


def check_clipped(got, grads, norm, max_norm):
    factor = ff.clip_factor(norm, max_norm)
    for o, g in zip(got, grads):
        ref = f64(g) * factor
        if factor == 1.0:
            assert torch.equal(o, g)
            continue
        tol = (HALF[g.dtype] + 4 * U) * np.abs(ref) + LEAST[g.dtype]
        assert (np.abs(f64(o) - ref) <= tol).all()


SIZES = ([1], [7], [8], [2047, 1, 9], [2048], [2049, 0, 5], [3] * 113, [100000, 64, 64, 12345], [1] * 300,
         [int(v) for v in np.random.default_rng(0).integers(0, 5000, 230)], [5000011])


@pytest.mark.parametrize("kinds", [("f32",), ("bf16",), ("f16",), ("f32", "bf16", "f16")], ids="-".join)
@pytest.mark.parametrize("shift", [0, 1])
def test_norm_and_clip(kinds, shift):
    etpc = _etpc()
    for k, sizes in enumerate(SIZES):
        note(f"grad norm {kinds} shift={shift} tensors={len(sizes)} elements={sum(sizes)}")
        rng = np.random.default_rng(k)
        grads = tensors(rng, sizes, kinds, shift=shift)
        before = [g.clone() for g in grads]
        ref = ff.grad_norm([f64(g) for g in grads])
        check_norm(etpc.etpc_grad_norm(grads), ref)
        check_norm(etpc.etpc_grad_norm(grads, ord=math.inf), ff.grad_norm([f64(g) for g in grads], np.inf))
        for part in (0.3, 2.0):
            outs = tensors(rng, sizes, kinds, shift=1 - shift)
            check_norm(etpc.etpc_clip_grad_norm(grads, part * ref, outs=outs), ref)
            check_clipped(outs, before, ref, part * ref)
            assert all(torch.equal(a, b) for a, b in zip(grads, before))
        check_norm(etpc.etpc_clip_grad_norm(grads, 2 * ref + 1), ref)
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
        check_norm(etpc.etpc_clip_grad_norm(grads, 0.3 * ref), ref)
        check_clipped(grads, before, ref, 0.3 * ref)
        assert all(shift == 0 or float(g._base[0]) == 0 for g in grads)   # what lies before a tensor


def test_empty_lists():
    etpc = _etpc()
    assert float(etpc.etpc_grad_norm([])) == 0 and float(etpc.etpc_clip_grad_norm([], 1.0)) == 0
    none = torch.zeros(0, device="cuda")
    assert float(etpc.etpc_grad_norm([none])) == 0 and float(etpc.etpc_clip_grad_norm([none, none], 1.0)) == 0


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_not_finite(kind, bad):
    """The norm tells, and the gradients stay as they are."""
    etpc = _etpc()
    rng = np.random.default_rng(2)
    for where in (0, 4999):
        grads = tensors(rng, [5000, 70], [kind])
        grads[0][where] = bad
        before = [g.clone() for g in grads]
        outs = [torch.zeros_like(g) for g in grads]
        for ord in (2, math.inf):
            norm = float(etpc.etpc_grad_norm(grads, ord=ord))
            assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
            norm = float(etpc.etpc_clip_grad_norm(grads, 0.1, ord=ord, outs=outs))
            assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
            etpc.etpc_clip_grad_norm(grads, 0.1, ord=ord)
            for a in (grads, outs):
                assert all(torch.equal(x.nan_to_num(7), y.nan_to_num(7)) for x, y in zip(a, before))


def test_range():
    """Squares past fp32's range and below its smallest number."""
    etpc = _etpc()
    big = torch.full((1000,), 1e30, device="cuda")
    check_norm(etpc.etpc_grad_norm([big]), float(np.float32(1e30)) * math.sqrt(1000))
    check_norm(etpc.etpc_clip_grad_norm([big], 1.0), float(np.float32(1e30)) * math.sqrt(1000))
    check_norm(etpc.etpc_grad_norm([big]), 1.0)
    small = torch.full((999,), 1e-30, device="cuda")
    check_norm(etpc.etpc_grad_norm([small]), float(np.float32(1e-30)) * math.sqrt(999))
    most = torch.full((4,), 3e38, device="cuda")
    assert float(etpc.etpc_clip_grad_norm([most], 1.0)) == math.inf and float(most[0]) == float(np.float32(3e38))


def test_dense_layouts():
    etpc = _etpc()
    w = torch.randn(40, 30, device="cuda").t()
    p = torch.randn(3, 4, 5, device="cuda").permute(2, 0, 1)
    ref = ff.grad_norm([f64(w), f64(p)])
    check_norm(etpc.etpc_grad_norm([w, p]), ref)
    before = [w.clone(), p.clone()]
    check_norm(etpc.etpc_clip_grad_norm([w, p], 0.5 * ref), ref)
    check_clipped([w, p], before, ref, 0.5 * ref)
    with pytest.raises(ValueError, match="block of memory"):
        etpc.etpc_grad_norm([torch.randn(8, 8, device="cuda")[:, :4]])
    with pytest.raises(etpc.EtpcError, match="overlap"):
        etpc.etpc_clip_grad_norm([before[0], before[0]], 1.0)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_ends_in_place(kind):
    """In place the same bits as into other tensors, wherever the last vector of a tensor ends and whichever wave has it."""
    etpc = _etpc()
    rng = np.random.default_rng(13)
    sizes = [base + end for base in (0, 8, 512, 2040, 2048, 8184) for end in range(8) if base + end]
    grads = tensors(rng, sizes, [kind], shift=1)
    before = [g.clone() for g in grads]
    outs = [torch.zeros_like(g) for g in grads]
    ref = ff.grad_norm([f64(g) for g in grads])
    for _ in range(5):
        for g, b in zip(grads, before):
            g.copy_(b)
        check_norm(etpc.etpc_clip_grad_norm(grads, 0.3 * ref, outs=outs), ref)
        check_norm(etpc.etpc_clip_grad_norm(grads, 0.3 * ref), ref)
        assert all(torch.equal(g, o) for g, o in zip(grads, outs))
    check_clipped(grads, before, ref, 0.3 * ref)
