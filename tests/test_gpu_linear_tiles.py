"""GPU checks of the dense layer's tiles at sizes that test_gpu_linear.py does not reach; oracle and tolerances are
those of that file."""
import pytest
import torch

from tests.test_gpu_linear import run_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("kind,rows,n_in,n_out,layout,pitch", [
    ("f32", 4097, 512, 256, "io", 0), ("f32", 4098, 512, 256, "oi", 5), ("f32", 4099, 512, 256, "io", 0), ("f32", 6146, 136, 512, "io", 0),
    ("f32", 8193, 260, 260, "oi", 0), ("bf16", 16385, 264, 2048, "io", 8), ("f16", 16386, 264, 2040, "oi", 0),
    ("bf16", 16387, 264, 2048, "io", 0), ("f16", 2049, 512, 512, "io", 8)])
def test_rows_past_the_last_tile(kind, rows, n_in, n_out, layout, pitch):
    """One or two of them, where they go to the kernel for few rows and where they stay a tile; three."""
    run_case(rows, rows, n_in, n_out, kind, "silu", layout, pitch)
