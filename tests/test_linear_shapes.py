"""Shapes of the dense layer's products (no GPU): the ranges of k cover it whatever its length."""
import ctypes as C

import pytest

import equivariant_gnn_tensor_amd as etpc


class Args(C.Structure):   # MatmulArgs
    _fields_ = [(n, C.c_void_p) for n in ("a", "b", "c", "z", "res", "bias", "part")] + \
        [(n, C.c_int64) for n in ("lda", "ldb", "ldc", "ldz", "ldres")] + \
        [(n, C.c_int32) for n in ("M", "N", "K", "k_split", "splits", "act", "tiles_m", "tiles_n")]


class Shape(C.Structure):   # MatmulShape
    _fields_ = [(n, C.c_int) for n in ("tile", "grain", "splits", "k_split", "stages")]


ROWS_COLS, COLS_COLS = 0, 2
matmul_shape = getattr(etpc.lib, "_ZN4etpc12matmul_shapeERKNS_10MatmulArgsENS_10MatmulFormEib")
matmul_shape.argtypes, matmul_shape.restype = [C.POINTER(Args), C.c_int, C.c_int, C.c_bool], Shape
LONG = (1, 63, 64, 127, 128, 4097, 65408, (1 << 24) + 1, (1 << 31) - 65, (1 << 31) - 64, (1 << 31) - 2, (1 << 31) - 1)


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("sums", [False, True])
def test_ranges_cover_k(dtype, sums):
    """Every range starts inside k and together they end at or past its end; their starts stay within 31 bits."""
    for k in LONG if sums else (n for n in LONG if n <= 1 << 30):
        for m, n in ((3, 1), (64, 64), (129, 1), (776, 336), (64, 32768), (4096, 4096), (16448, 1)):
            s = matmul_shape(Args(lda=m if sums else k, ldb=n, M=m, N=n, K=k), COLS_COLS if sums else ROWS_COLS, dtype, sums)
            assert s.splits >= 1 and s.k_split >= 1
            assert s.splits * s.k_split >= k, (k, m, n, s.splits, s.k_split)
            assert (s.splits - 1) * s.k_split < k
