"""GPU checks of the dense layer's tiles at sizes that test_gpu_linear.py does not reach; oracle and tolerances are
those of that file."""
import numpy as np
import pytest
import torch

from tests.test_gpu_linear import KINDS, check_backward, check_forward, f64, matrix, run_case, vector, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _etpc():
    import equivariant_gnn_tensor_amd as etpc
    return etpc


@pytest.mark.parametrize("kind,rows,n_in,n_out,layout,pitch", [
    ("f32", 4097, 512, 256, "io", 0), ("f32", 4098, 512, 256, "oi", 5), ("f32", 4099, 512, 256, "io", 0), ("f32", 6146, 136, 512, "io", 0),
    ("f32", 8193, 260, 260, "oi", 0), ("bf16", 16385, 264, 2048, "io", 8), ("f16", 16386, 264, 2040, "oi", 0),
    ("bf16", 16387, 264, 2048, "io", 0), ("f16", 2049, 512, 512, "io", 8)])
def test_rows_past_the_last_tile(kind, rows, n_in, n_out, layout, pitch):
    """One or two of them, where they go to the kernel for few rows and where they stay a tile; three."""
    run_case(rows, rows, n_in, n_out, kind, "silu", layout, pitch)


def for_kinds(*case):
    return [(kind, *case) for kind in KINDS]


# Whole 16-byte pieces, even rows, odd rows: loads of 16 and 4 bytes and through registers, either layout.  First many
# rows to few outputs, then few rows to many, so that each tile has more of them than are resident and walks on.
WALKING = (for_kinds(82000, 136, 40, "io", 0) + for_kinds(82000, 136, 40, "oi", 0) + for_kinds(82001, 134, 38, "io", 0)
           + for_kinds(82001, 134, 38, "oi", 0) + for_kinds(82000, 135, 37, "io", 0) + for_kinds(82000, 135, 37, "oi", 0)
           + for_kinds(130, 40, 82000, "io", 0) + for_kinds(130, 40, 82000, "oi", 0) + for_kinds(130, 38, 82002, "io", 0)
           + for_kinds(130, 38, 82002, "oi", 0) + for_kinds(130, 37, 82001, "io", 0) + for_kinds(130, 37, 82001, "oi", 0)
           + for_kinds(130, 72, 66000, "io", 0) + for_kinds(130, 70, 66002, "oi", 0) + for_kinds(130, 71, 66001, "io", 0))


@pytest.mark.parametrize("kind,rows,n_in,n_out,layout,pitch", WALKING)
def test_tiles_that_walk_on(kind, rows, n_in, n_out, layout, pitch):
    run_case(rows + n_out, rows, n_in, n_out, kind, "silu", layout, pitch, residual=layout == "io")


@pytest.mark.parametrize("kind,rows,n_in,n_out,layout,pitch", [
    ("bf16", 136, 264, 66400, "io", 0), ("bf16", 136, 264, 66400, "oi", 8), ("f16", 136, 264, 66400, "io", 8),
    ("f16", 136, 264, 66400, "oi", 0)])
def test_large_tiles_that_walk_on(kind, rows, n_in, n_out, layout, pitch):
    run_case(rows + n_out, rows, n_in, n_out, kind, "silu", layout, pitch)


@pytest.mark.parametrize("kind,rows,n_in,n_out,layout,pitch", (
    for_kinds(8200, 264, 520, "io", 0) + for_kinds(8200, 264, 520, "oi", 5) + for_kinds(8200, 262, 518, "io", 0)
    + for_kinds(8200, 264, 520, "io", 5)))
def test_weight_gradients_on_middle_tiles(kind, rows, n_in, n_out, layout, pitch):
    run_case(rows, rows, n_in, n_out, kind, "silu", layout, pitch)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,n_in,n_out", [(82000, 135, 37), (130, 40, 82000), (8200, 264, 520), (130, 72, 66000)])
def test_repeated_rows_on_every_tile(kind, rows, n_in, n_out):
    """One row for all goes through registers in fp32 too."""
    etpc = _etpc()
    rng = np.random.default_rng(rows)
    w, b = weights(rng, n_in, n_out, kind, "oi"), vector(rng, n_out)
    x, y_bar = (matrix(rng, 1, n, kind).expand(rows, n) for n in (n_in, n_out))
    y, _ = etpc.etpc_linear(x, w, b)
    check_forward(y, None, f64(x), f64(w), f64(b), None, "none", kind)
    x_bar, w_bar, b_bar = etpc.etpc_linear_backward(x, w, y_bar)
    # fp16 ends at 65504 and rounds what is 65520 or more to an infinity: such sums (rows x y_bar, up to 82000 times a product
    # of two numbers) are right as infinities of their sign, where the exact one reaches 65520 within the tolerance (below
    # 1 % of it: steps(82000) + 2^-11 = 0.54 %).
    exact = torch.from_numpy(f64(x).T @ f64(y_bar)).cuda()
    past = torch.isinf(w_bar)
    assert bool((1.01 * exact.abs()[past] >= 65520).all()) and (kind == "f16" or not past.any())
    assert torch.equal(torch.sign(w_bar[past]).double(), torch.sign(exact[past]))
    check_backward(x_bar, torch.where(past, exact, w_bar.double()), b_bar, f64(x), f64(w), f64(y_bar), None, "none", kind)


@pytest.mark.parametrize("kind,rows,n_in,n_out,layout,pitch", (
    for_kinds(90001, 64, 64, "io", 0) + for_kinds(90007, 62, 62, "oi", 5) + for_kinds(81921, 62, 62, "io", 0) + for_kinds(81920, 62, 62, "io", 0)
    + for_kinds(90033, 128, 32, "oi", 0) + for_kinds(90002, 127, 31, "io", 8) + for_kinds(65537, 32, 128, "io", 0)
    + for_kinds(65540, 31, 99, "oi", 5) + for_kinds(65600, 50, 75, "io", 0) + for_kinds(65599, 50, 80, "oi", 0)
    + for_kinds(90020, 90, 50, "io", 8) + for_kinds(90064, 48, 56, "oi", 8) + for_kinds(65536, 31, 99, "io", 0)
    + for_kinds(65545, 33, 70, "io", 0)))
def test_narrow_rows_past_a_round_of_tiles(kind, rows, n_in, n_out, layout, pitch):
    """On either side of each limit past which a narrow layer takes the kernel that keeps its weights in LDS."""
    run_case(rows, rows, n_in, n_out, kind, "gelu" if n_in % 2 else "tanh", layout, pitch)
