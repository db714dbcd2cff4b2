"""GPU checks of the node-wise operators against oracle/nodewise.py (float64).

Tolerances, u = 2^-24.  Inputs reach the oracle exactly (already rounded to the element
type).  A row's sums add at most 64 numbers one after another (32 in a lane, then trees),
so a mean is off by at most 64 u times the row's largest magnitude; a sum over rows adds at
most 512 one after another.  Each result carries a few roundings of its own terms (counted
as 64 u of their magnitudes as well) and one rounding to the element type: half a unit,
2^-9 (bf16) and 2^-12 (fp16) of the value, counted as 2^-8 and 2^-11 to cover a neighbour
reached through the first error; fp16's smallest step is 2^-24.
"""
import numpy as np
import pytest
import torch

from oracle import nodewise as nw
from oracle.wigner import random_rotation
from tests.gpu_helpers import note
from tests.test_oracle_nodewise import DIM, IRREPS, rotate

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {"f32": U, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEAST = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}
ROW_TERMS, COL_TERMS = 64 * U, 512 * U
EPS = 1e-5
COLS = (1, 2, 5, 8, 9, 16, 31, 64, 65, 128, 200, 256, 257, 512, 577, 1024, 1025, 2047, 2048, 2049, 4096, 4100, 8192,
        8200, 16384, 16385, 20000)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _etpc():
    import equivariant_gnn_tensor_amd as etpc
    return etpc


def f64(t):
    return t.detach().double().cpu().numpy()


def tensor(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def rows(rng, n, cols, dtype, pitch=None, shift=0.5):
    """A [n, cols] view of rows `pitch` elements apart; every other element is NaN."""
    pitch = pitch or cols
    full = torch.full((n, pitch), float("nan"), dtype=DTYPES[dtype], device="cuda")
    full[:, :cols] = tensor(rng.standard_normal((n, cols)) * rng.uniform(0.3, 2.0, (n, 1)) + shift, DTYPES[dtype])
    return full[:, :cols]


def close(got, ref, bound, what, kind="f32"):
    """|got - ref| <= bound + the rounding of the result; equal where ref is not finite."""
    got = f64(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    tol = bound + ROUND[kind] * np.abs(ref) + LEAST[kind]
    bad = ~(np.abs(got - ref) <= tol) & np.isfinite(ref)
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], np.broadcast_to(tol, ref.shape)[bad][:4])
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what


def check_forward(y, mean, rstd, h, h_err, w, b, kind):
    """Forward results for the float64 rows h, which the kernel holds to within h_err."""
    ry, rm, rs = nw.layer_norm(h, w, b, EPS)
    top = np.abs(h).max(axis=1) if h.size else np.zeros(0)
    d_mean = ROW_TERMS * top + h_err
    close(mean, rm, d_mean, "mean")
    # the centred numbers are off by their own rounding and d_mean; a shift of all of them
    # changes the variance by its square only
    rel = ROW_TERMS + (d_mean * rs) ** 2 + 2 * h_err * rs
    close(rstd, rs, rel * rs, "rstd")
    xh = (h - rm[:, None]) * rs[:, None]
    err = np.abs(w) * (rs * d_mean)[:, None] + (rel[:, None] + ROW_TERMS) * np.abs(w * xh) + ROW_TERMS * np.abs(b)
    close(y, ry, err, "y", kind)


def check_backward(x_bar, w_bar, b_bar, x, y_bar, mean, rstd, w, kind, extra=None):
    rx, rw, rb = nw.layer_norm_backward(x, y_bar, mean, rstd, w)
    xh = (x - mean[:, None]) * rstd[:, None]
    g = y_bar * w
    err = ROW_TERMS * rstd[:, None] * (np.abs(g) + np.abs(g).mean(1, keepdims=True)
                                       + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
    if extra is not None:
        rx, err = rx + extra, err + ROW_TERMS * np.abs(extra)
    if x_bar is not None:
        close(x_bar, rx, err, "x_bar", kind)
    if w_bar is not None:
        close(w_bar, rw, COL_TERMS * np.abs(y_bar * xh).sum(0), "w_bar")
    if b_bar is not None:
        close(b_bar, rb, COL_TERMS * np.abs(y_bar).sum(0), "b_bar")
    return rx, err


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [1, 3, 70])
def test_layer_norm(kind, n):
    etpc = _etpc()
    rng = np.random.default_rng(100 + n)
    for cols in COLS:
        note(f"layer norm {kind} rows={n} cols={cols}")
        x, yb = rows(rng, n, cols, kind), rows(rng, n, cols, kind, shift=0.0)
        w, b = tensor(rng.standard_normal(cols)), tensor(rng.standard_normal(cols))
        y, mean, rstd = etpc.etpc_layer_norm(x, w, b, eps=EPS)
        check_forward(y, mean, rstd, f64(x), np.zeros(n), f64(w), f64(b), kind)
        x_bar, w_bar, b_bar = etpc.etpc_layer_norm_backward(x, yb, mean, rstd, w)
        check_backward(x_bar, w_bar, b_bar, f64(x), f64(yb), f64(mean), f64(rstd), f64(w), kind)


@pytest.mark.parametrize("kind,n,cols", [("f32", 5000, 64), ("bf16", 3001, 577), ("f16", 2500, 1024), ("f32", 20011, 3),
                                         ("bf16", 1100, 4104), ("f16", 3000, 1), ("f32", 300, 16400)])
def test_layer_norm_many_rows(kind, n, cols):
    """More rows than workgroups: groups walk several rows and the column sums take two stages."""
    etpc = _etpc()
    rng = np.random.default_rng(n)
    note(f"layer norm {kind} rows={n} cols={cols}")
    x, yb = rows(rng, n, cols, kind), rows(rng, n, cols, kind, shift=0.0)
    w, b = tensor(rng.standard_normal(cols)), tensor(rng.standard_normal(cols))
    y, mean, rstd = etpc.etpc_layer_norm(x, w, b, eps=EPS)
    check_forward(y, mean, rstd, f64(x), np.zeros(n), f64(w), f64(b), kind)
    outs = etpc.etpc_layer_norm_backward(x, yb, mean, rstd, w)
    check_backward(*outs, f64(x), f64(yb), f64(mean), f64(rstd), f64(w), kind)
    again = etpc.etpc_layer_norm_backward(x, yb, mean, rstd, w)
    assert all(torch.equal(p, q) for p, q in zip(outs, again))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("cols,pitch,first", [(64, 576, 64), (64, 77, 3), (33, 40, 1), (130, 131, 1), (1024, 1031, 7),
                                              (2500, 2501, 1)])
def test_layer_norm_strided_views(kind, cols, pitch, first):
    """A block of columns of wider rows, read and written in place of its rows: neighbours stay
    as they are, odd offsets misalign every row."""
    etpc = _etpc()
    rng = np.random.default_rng(cols)
    n = 37
    note(f"strided layer norm {kind} cols={cols} pitch={pitch} first={first}")
    big = torch.full((n, pitch + first), float("nan"), dtype=DTYPES[kind], device="cuda")
    x = big[:, first:first + cols]
    x.copy_(tensor(rng.standard_normal((n, cols)) + 0.3, DTYPES[kind]))
    out = torch.full((n, pitch + first), 7.0, dtype=DTYPES[kind], device="cuda")
    y = out[:, first:first + cols]
    yb = rows(rng, n, cols, kind, pitch=cols + 3, shift=0.0)
    w, b = tensor(rng.standard_normal(cols)), tensor(rng.standard_normal(cols))
    got, mean, rstd = etpc.etpc_layer_norm(x, w, b, eps=EPS, y=y)
    assert got is y
    check_forward(y, mean, rstd, f64(x), np.zeros(n), f64(w), f64(b), kind)
    x_bar = out[:, first:first + cols]
    wb, bb = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    etpc.etpc_layer_norm_backward(x, yb, mean, rstd, w, outs=(x_bar, wb, bb))
    check_backward(x_bar, wb, bb, f64(x), f64(yb), f64(mean), f64(rstd), f64(w), kind)
    assert (out[:, :first] == 7).all() and (out[:, first + cols:] == 7).all()


def test_outputs_between_the_columns_of_inputs():
    """Columns of one tensor's rows as input and output: their rows interleave in memory without
    meeting, which is no overlap; a dropout works in place on such a view."""
    etpc = _etpc()
    rng = np.random.default_rng(9)
    big = tensor(rng.standard_normal((23, 150)))
    before = big.clone()
    x, y = big[:, :64], big[:, 64:128]
    _, mean, rstd = etpc.etpc_layer_norm(x, y=y, eps=EPS)
    check_forward(y, mean, rstd, f64(before[:, :64]), np.zeros(23), np.ones(64), np.zeros(64), "f32")
    assert torch.equal(big[:, :64], before[:, :64]) and torch.equal(big[:, 128:], before[:, 128:])
    with pytest.raises(etpc.EtpcError, match="overlap"):
        etpc.etpc_layer_norm(big[:, :64], y=big[:, 63:127])
    tail = big[:, 128:147]
    etpc.etpc_dropout(tail, 0.4, 5, 6, y=tail)
    ref = nw.dropout(f64(before[:, 128:147]), 0.4, 5, 6)
    close(tail, ref, U * np.abs(ref), "y")
    assert torch.equal(big[:, :64], before[:, :64]) and torch.equal(big[:, 147:], before[:, 147:])


def test_layer_norm_broadcast_rows_and_shapes():
    """An expanded row (stride 0) is read for every row; leading axes are rows."""
    etpc = _etpc()
    rng = np.random.default_rng(5)
    x = rows(rng, 1, 200, "f32").expand(41, 200)
    y, mean, rstd = etpc.etpc_layer_norm(x, eps=EPS)
    check_forward(y, mean, rstd, f64(x), np.zeros(41), np.ones(200), np.zeros(200), "f32")
    x3 = rows(rng, 12, 40, "f32").reshape(3, 4, 40)
    y3, m3, r3 = etpc.etpc_layer_norm(x3, eps=EPS)
    assert y3.shape == (3, 4, 40) and m3.shape == r3.shape == (3, 4)
    check_forward(y3.reshape(12, 40), m3.reshape(12), r3.reshape(12), f64(x3).reshape(12, 40), np.zeros(12), np.ones(40),
                  np.zeros(40), "f32")
    yb = rows(rng, 1, 40, "f32").expand(3, 4, 40)
    xb, wb, bb = etpc.etpc_layer_norm_backward(x3, yb, m3, r3)
    check_backward(xb.reshape(12, 40), wb, bb, f64(x3).reshape(12, 40), f64(yb).reshape(12, 40), f64(m3).reshape(12),
                   f64(r3).reshape(12), np.ones(40), "f32")
    assert etpc.etpc_layer_norm(torch.zeros(0, 8, device="cuda"))[0].shape == (0, 8)
    _, wb, bb = etpc.etpc_layer_norm_backward(torch.zeros(0, 8, device="cuda"), torch.zeros(0, 8, device="cuda"),
                                              torch.zeros(0, device="cuda"), torch.zeros(0, device="cuda"))
    assert (wb == 0).all() and (bb == 0).all()


def test_layer_norm_hard_rows():
    """Constant rows, a mean far above the spread, tiny and huge rows; a row with an infinity or
    a NaN spoils itself and the sums over rows, no other row."""
    etpc = _etpc()
    rng = np.random.default_rng(6)
    cols = 600
    x = rng.standard_normal((7, cols))
    x[0] = 3.25
    x[1] += 4096.0
    x[2] *= 1e-12
    x[3] *= 1e15
    x[4] = 0.0
    x = tensor(x)
    y, mean, rstd = etpc.etpc_layer_norm(x, eps=EPS)
    check_forward(y, mean, rstd, f64(x), np.zeros(7), np.ones(cols), np.zeros(cols), "f32")
    assert (y[4] == 0).all()
    bad = x.clone()
    bad[5, 77], bad[6, 3] = float("inf"), float("nan")
    y2, _, _ = etpc.etpc_layer_norm(bad, eps=EPS)
    assert torch.equal(y2[:5], y[:5]) and torch.isnan(y2[5:]).all()
    # eps = 0 on a constant row is 0 * inf
    assert torch.isnan(etpc.etpc_layer_norm(x, eps=0.0)[0][0]).all()


@pytest.mark.parametrize("level", [0.0, 300.0, 1e5])
def test_rows_far_from_zero(level):
    """The mean is corrected by what is left after it, so the centred numbers d are off by 64 u
    of their own size (the sum of what is left) whatever the level: exact differences of
    numbers near each other.  Held to that, with 64 u of the result and its level's rounding
    for the stored mean."""
    etpc = _etpc()
    rng = np.random.default_rng(10)
    for n, cols in ((40, 700), (3, 64), (2, 3000), (2, 18000)):
        x = tensor(level + rng.standard_normal((n, cols)))
        for y, mean, rstd in (etpc.etpc_layer_norm(x, eps=EPS),
                              (lambda y, st: (y, st[:, 0, 0], st[:, 0, 1]))(*etpc.etpc_irreps_norm(f"{cols}x0e", x, eps=EPS))):
            ry, rm, rs = nw.layer_norm(f64(x), np.ones(cols), np.zeros(cols), EPS)
            top = np.abs(ry).max(axis=1)
            # the irreps norm's segments past 512 numbers add up to 256 numbers in a lane
            terms = 64 * U if cols <= 512 else 320 * U
            assert (np.abs(f64(y) - ry) <= 2 * terms * top[:, None] + terms * np.abs(ry)).all()
            assert (np.abs(f64(mean) - rm) <= terms * top / rs + 2 * U * np.abs(rm)).all()
            assert (np.abs(f64(rstd) - rs) <= 2 * terms * rs).all()


def test_layer_norm_wanted_outputs():
    etpc = _etpc()
    rng = np.random.default_rng(7)
    x, yb = rows(rng, 50, 96, "f32"), rows(rng, 50, 96, "f32", shift=0.0)
    w = tensor(rng.standard_normal(96))
    y, none1, none2 = etpc.etpc_layer_norm(x, w, stats=False)
    y2, mean, rstd = etpc.etpc_layer_norm(x, w)
    assert none1 is None and none2 is None and torch.equal(y, y2)
    full = etpc.etpc_layer_norm_backward(x, yb, mean, rstd, w)
    for want in (("x",), ("w",), ("b",), ("w", "b"), ("x", "b"), ()):
        part = etpc.etpc_layer_norm_backward(x, yb, mean, rstd, w, want=want)
        for name, p, q in zip("xwb", part, full):
            assert (p is None) if name not in want else torch.equal(p, q)


def test_gradients_against_differences():
    """Central differences of the float64 forward map at the kernel's own inputs."""
    etpc = _etpc()
    rng = np.random.default_rng(8)
    n, cols, p, seed, off = 2, 19, 0.3, 11, 12
    x, res = rows(rng, n, cols, "f32"), rows(rng, n, cols, "f32")
    yb, hb = rows(rng, n, cols, "f32", shift=0.0), rows(rng, n, cols, "f32", shift=0.0)
    w, b = tensor(rng.standard_normal(cols)), tensor(rng.standard_normal(cols))
    y, h, mean, rstd = etpc.etpc_dropout_add_layer_norm(x, res, w, b, p=p, seed=seed, offset=off, eps=EPS)
    got = etpc.etpc_dropout_add_layer_norm_backward(h, yb, mean, rstd, w, h_bar=hb, p=p, seed=seed, offset=off)
    base = [f64(t) for t in (x, res, w, b)]

    def loss(v):
        hh = v[1] + nw.dropout(v[0], p, seed, off)
        return (f64(yb) * nw.layer_norm(hh, v[2], v[3], EPS)[0]).sum() + (f64(hb) * hh).sum()

    for k, name in enumerate(("x_bar", "residual_bar", "w_bar", "b_bar")):
        for i in np.ndindex(base[k].shape):
            up, down = [v.copy() for v in base], [v.copy() for v in base]
            up[k][i] += 1e-5
            down[k][i] -= 1e-5
            diff = (loss(up) - loss(down)) / 2e-5
            # 1e-7 of the differences, 64 u of sums of terms of magnitude up to about 20
            assert abs(float(got[k][i]) - diff) < 1e-7 + 64 * U * 20, (name, i)


# ---------------------------------------------------------------- dropout

@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,cols,pitch", [(1, 1, 1), (1, 4096, 4096), (5, 7, 7), (64, 64, 64), (33, 100, 107), (1000, 8, 8),
                                          (3001, 3, 3), (17, 1001, 1002), (2, 70001, 70001)])
def test_dropout(kind, n, cols, pitch):
    etpc = _etpc()
    rng = np.random.default_rng(n + cols)
    x = rows(rng, n, cols, kind, pitch=pitch)
    for p, seed, off in ((0.1, 1, 0), (0.75, (1 << 63) + 12345, (1 << 40) + 7), (0.0, 3, 4), (1e-7, 3, 4), (1.0, 5, 6)):
        note(f"dropout {kind} {n}x{cols} p={p}")
        y = etpc.etpc_dropout(x, p, seed, off)
        ref = nw.dropout(f64(x), p, seed, off)
        close(y, ref, U * np.abs(ref), "y", kind)
        assert np.array_equal(f64(y) == 0, ref == 0)
        inplace = x.clone()
        assert etpc.etpc_dropout(inplace, p, seed, off, y=inplace) is inplace and torch.equal(inplace, y)
    assert torch.equal(etpc.etpc_dropout(x, 0.0, 1), x)


def test_dropout_leaves_no_trace_of_dropped_values():
    """Infinities and NaN in dropped places become 0; with p = 1 every row is empty."""
    etpc = _etpc()
    n, cols, p, seed = 20, 333, 0.4, 9
    keep = nw.keep_fields(n, (cols + 7) // 8, p, seed, 2)[:, :cols]
    x = torch.ones(n, cols, device="cuda")
    x[torch.from_numpy(~keep).cuda()] = float("inf")
    y = etpc.etpc_dropout(x, p, seed, 2)
    assert torch.isfinite(y).all() and np.array_equal(f64(y) != 0, keep)
    res = torch.randn(n, cols, device="cuda")
    nan = torch.full((n, cols), float("nan"), device="cuda")
    y, h, mean, rstd = etpc.etpc_dropout_add_layer_norm(nan, res, p=1.0, seed=1)
    assert torch.equal(h, res)
    check_forward(y, mean, rstd, f64(res), np.zeros(n), np.ones(cols), np.zeros(cols), "f32")
    y, h, _, _ = etpc.etpc_dropout_add_layer_norm(nan, None, p=1.0, seed=1)
    assert (h == 0).all() and (y == 0).all()
    xb, rb, _, _ = etpc.etpc_dropout_add_layer_norm_backward(h, res, torch.zeros(n, device="cuda"),
                                                             torch.ones(n, device="cuda"), p=1.0, seed=1)
    assert (xb == 0).all() and (rb != 0).any()


def test_dropout_offsets_past_32_bits():
    """Rows 2^31 elements apart and more: element offsets need 64 bits."""
    etpc = _etpc()
    stride, cols, n = (1 << 31) + 8, 100, 3
    buf = torch.zeros(2 * stride + cols, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((n, cols), (stride, 1))
    x.copy_(torch.randn(n, cols, device="cuda"))
    note("rows past 2^31 elements")
    y = etpc.etpc_dropout(x, 0.25, 3, 4)
    ref = nw.dropout(f64(x), 0.25, 3, 4)
    close(y, ref, U * np.abs(ref), "y", "bf16")
    z, mean, rstd = etpc.etpc_layer_norm(x, eps=EPS)
    check_forward(z, mean, rstd, f64(x), np.zeros(n), np.ones(cols), np.zeros(cols), "bf16")
    xb, _, _ = etpc.etpc_layer_norm_backward(x, y, mean, rstd)
    check_backward(xb, None, None, f64(x), f64(y), f64(mean), f64(rstd), np.ones(cols), "bf16")


# ---------------------------------------------------------------- the join

@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,cols", [(1, 1024), (3, 5), (70, 64), (41, 577), (9, 2047), (6, 4097), (3, 9000), (2, 17001),
                                    (2600, 40)])
def test_join(kind, n, cols):
    etpc = _etpc()
    rng = np.random.default_rng(cols)
    note(f"join {kind} {n}x{cols}")
    x, res = rows(rng, n, cols, kind, pitch=cols + 5), rows(rng, n, cols, kind)
    yb, hb = rows(rng, n, cols, kind, shift=0.0), rows(rng, n, cols, kind, pitch=cols + 2, shift=0.0)
    w, b = tensor(rng.standard_normal(cols)), tensor(rng.standard_normal(cols))
    p, seed, off = 0.2, 77, (1 << 33) + 5
    for r, q in ((res, p), (None, p), (res, 0.0)):
        y, h, mean, rstd = etpc.etpc_dropout_add_layer_norm(x, r, w, b, p=q, seed=seed, offset=off, eps=EPS)
        dropped = nw.dropout(f64(x), q, seed, off)
        rh = dropped + (f64(r) if r is not None else 0.0)
        h_err = 3 * U * (np.abs(dropped) + np.abs(rh))
        close(h, rh, h_err, "h", kind)
        check_forward(y, mean, rstd, rh, h_err.max(axis=1), f64(w), f64(b), kind)
        if q == 0.0 or r is None:
            continue
        for extra in (hb, None):
            xb, rb, wb, bb = etpc.etpc_dropout_add_layer_norm_backward(h, yb, mean, rstd, w, h_bar=extra, p=q, seed=seed,
                                                                       offset=off)
            rx, err = check_backward(rb, wb, bb, f64(h), f64(yb), f64(mean), f64(rstd), f64(w), kind,
                                     extra=f64(extra) if extra is not None else None)
            scale = 65536.0 / (65536 - nw.threshold(q))
            close(xb, nw.dropout(rx, q, seed, off), scale * (err + U * np.abs(rx)), "x_bar", kind)
            only = etpc.etpc_dropout_add_layer_norm_backward(h, yb, mean, rstd, w, h_bar=extra, p=q, seed=seed, offset=off,
                                                             want=("x",))
            assert torch.equal(only[0], xb) and only[1:] == (None, None, None)


def test_join_without_residual_and_dropout_is_the_layer_norm():
    etpc = _etpc()
    x = rows(np.random.default_rng(1), 33, 300, "bf16")
    y, mean, rstd = etpc.etpc_layer_norm(x)
    y2, h, mean2, rstd2 = etpc.etpc_dropout_add_layer_norm(x, None)
    assert torch.equal(y, y2) and torch.equal(h, x) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)


# ---------------------------------------------------------------- irreps features

IRREP_LISTS = ["8x0e+8x1o", "1x0e", "1x3o", "5x0o+3x1o+7x2e+2x3o+9x0e", "64x0e+64x1o+64x2e+64x3o", "128x0e+100x1e",
               "300x3e+2x0e", "2049x0e+1x1o", "700x3o+2100x0e", "+".join(["4x0e"] * 64)]


def _parsed(text):
    etpc = _etpc()
    ir = etpc.parse_irreps(text)
    d = etpc.etpc_irreps_dims(text)
    return ir, d["dim"], d["channels"], d["biases"]


@pytest.mark.parametrize("text", IRREP_LISTS)
@pytest.mark.parametrize("n", [1, 6, 2500])
def test_irreps_norm(text, n):
    etpc = _etpc()
    ir, dim, channels, biases = _parsed(text)
    if n * dim > 3_000_000:
        n = 400
    note(f"irreps norm {text[:40]} nodes={n}")
    rng = np.random.default_rng(n + dim)
    x, yb = rows(rng, n, dim, "f32", shift=0.2), rows(rng, n, dim, "f32", shift=0.0)
    w, b = tensor(rng.standard_normal(channels)), tensor(rng.standard_normal(biases))
    y, stats = etpc.etpc_irreps_norm(text, x, w, b, eps=EPS)
    wb_full = etpc.etpc_irreps_norm_backward(text, x, yb, stats, w)
    X, Y, W, B = f64(x), f64(yb), f64(w), f64(b)
    ry, rs = nw.irreps_norm(X, ir, W, B, EPS)
    rxb, rwb, rbb = nw.irreps_norm_backward(X, Y, f64(stats), ir, W)
    gx, gs, gy = f64(wb_full[0]), f64(stats), f64(y)
    # a lane adds at most 32 numbers (128 in segments past 2048 numbers) before the tree
    row_terms = 256 * U
    for k, (mul, l, parity, off, ch, bias) in enumerate(nw.blocks(ir)):
        part = slice(off, off + mul * (2 * l + 1))
        v, gain = X[:, part], np.tile(W[ch:ch + mul], 2 * l + 1)
        d_mean = row_terms * np.abs(v).max(axis=1) if l == 0 else np.zeros(n)
        mean, rstd = rs[:, k, 0], rs[:, k, 1]
        assert (np.abs(gs[:, k, 0] - mean) <= d_mean).all()
        rel = row_terms + (d_mean * rstd) ** 2
        assert (np.abs(gs[:, k, 1] - rstd) <= rel * rstd).all()
        xh = (v - mean[:, None]) * rstd[:, None]
        err = np.abs(gain) * (rstd * d_mean)[:, None] + (rel[:, None] + row_terms) * np.abs(gain * xh) + 4 * U * np.abs(ry[:, part])
        if bias is not None:
            err = err + 4 * U * np.abs(B[bias:bias + mul])
        assert (np.abs(gy[:, part] - ry[:, part]) <= err).all(), (k, "y")
        m, r = gs[:, k, 0][:, None], gs[:, k, 1][:, None]
        xh, g = (v - m) * r, Y[:, part] * gain
        err = row_terms * r * (np.abs(g) + np.abs(g).mean(1, keepdims=True) + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
        assert (np.abs(gx[:, part] - rxb[:, part]) <= err).all(), (k, "x_bar")
        # at most 512 nodes and 7 components one after another
        tol = 1024 * U * np.abs(Y[:, part] * xh).sum(0).reshape(2 * l + 1, mul).sum(0)
        assert (np.abs(f64(wb_full[1])[ch:ch + mul] - rwb[ch:ch + mul]) <= tol).all(), (k, "w_bar")
        if bias is not None:
            tol = 1024 * U * np.abs(Y[:, part]).sum(0)
            assert (np.abs(f64(wb_full[2])[bias:bias + mul] - rbb[bias:bias + mul]) <= tol).all(), (k, "b_bar")
    for want in (("x",), ("w", "b"), ("b",)):
        part = etpc.etpc_irreps_norm_backward(text, x, yb, stats, w, want=want)
        for name, p, q in zip("xwb", part, wb_full):
            assert (p is None) if name not in want else torch.equal(p, q)
    y2, none = etpc.etpc_irreps_norm(text, x, w, b, eps=EPS, keep_stats=False)
    assert none is None and torch.equal(y, y2)


@pytest.mark.parametrize("text", IRREP_LISTS)
@pytest.mark.parametrize("n", [1, 77])
def test_irreps_dropout(text, n):
    etpc = _etpc()
    ir, dim, _, _ = _parsed(text)
    x = rows(np.random.default_rng(dim), n, dim, "f32")
    for p, seed, off in ((0.3, 1, 2), (0.9, 1 << 50, 1 << 45), (0.0, 1, 2), (1.0, 1, 2)):
        note(f"irreps dropout {text[:40]} nodes={n} p={p}")
        y = etpc.etpc_irreps_dropout(text, x, p, seed, off)
        ref = nw.irreps_dropout(f64(x), ir, p, seed, off)
        close(y, ref, U * np.abs(ref), "y")
        assert np.array_equal(f64(y) == 0, ref == 0)
    again = x.clone()
    assert torch.equal(etpc.etpc_irreps_dropout(text, again, 0.3, 1, 2, y=again), etpc.etpc_irreps_dropout(text, x, 0.3, 1, 2))


def test_irreps_operators_commute_with_rotations():
    etpc = _etpc()
    rng = np.random.default_rng(3)
    x, R = rng.standard_normal((50, DIM)), random_rotation(rng)
    _, dim, channels, biases = _parsed(IRREPS)
    w, b = tensor(rng.standard_normal(channels)), tensor(rng.standard_normal(biases))
    for f in (lambda t: etpc.etpc_irreps_norm(IRREPS, tensor(t), w, b)[0],
              lambda t: etpc.etpc_irreps_dropout(IRREPS, tensor(t), 0.4, 5, 6)):
        # rounding of the rotated inputs and 64 u in the map, on numbers up to about 10
        assert np.abs(f64(f(rotate(x, R, True))) - rotate(f64(f(x)), R, True)).max() < 128 * U * 10


# ---------------------------------------------------------------- streams, graphs, refusals

def test_streams():
    """Work on a stream other than the current one, with outputs and workspace allocated there."""
    etpc = _etpc()
    x = torch.randn(5000, 200, device="cuda")
    yb = torch.randn(5000, 200, device="cuda")
    w = torch.randn(200, device="cuda")
    ref_y, mean, rstd = etpc.etpc_layer_norm(x, w)
    ref = etpc.etpc_layer_norm_backward(x, yb, mean, rstd, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y, m, r = etpc.etpc_layer_norm(x, w, stream=side)
    got = etpc.etpc_layer_norm_backward(x, yb, m, r, w, stream=side)
    d = etpc.etpc_dropout(y, 0.5, 1, 2, stream=side.cuda_stream)
    ir, stats = etpc.etpc_irreps_norm("50x0e+50x1o", x, stream=side)
    side.synchronize()
    assert torch.equal(y, ref_y) and all(torch.equal(p, q) for p, q in zip(got, ref))
    assert torch.equal(d, etpc.etpc_dropout(ref_y, 0.5, 1, 2))
    assert torch.equal(ir, etpc.etpc_irreps_norm("50x0e+50x1o", x)[0])


def test_graph_replays_with_a_device_offset():
    """A captured step reads the mask's offset on the device: replays with another offset give
    another mask, each equal to the eager call."""
    etpc = _etpc()
    n, cols, p, seed = 700, 320, 0.3, 21
    x, res = torch.randn(n, cols, device="cuda"), torch.randn(n, cols, device="cuda")
    yb = torch.randn(n, cols, device="cuda")
    w = torch.randn(cols, device="cuda")
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def run(offset):
        y, h, mean, rstd = etpc.etpc_dropout_add_layer_norm(x, res, w, p=p, seed=seed, offset=offset)
        return (y, h) + etpc.etpc_dropout_add_layer_norm_backward(h, yb, mean, rstd, w, p=p, seed=seed, offset=offset)

    run(step)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(step)
    for k in (5, 6, (1 << 41) + 3, 5):
        step.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        eager = run(k)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), k
    assert not torch.equal(run(5)[1], run(6)[1])


def test_binding_refusals():
    etpc = _etpc()
    x = torch.randn(6, 32, device="cuda")
    mean = rstd = torch.ones(6, device="cuda")
    for bad in (x.t(), x[:, ::2]):
        with pytest.raises(ValueError, match="contiguous"):
            etpc.etpc_layer_norm(bad)
    with pytest.raises(ValueError, match="leading axes"):
        etpc.etpc_layer_norm(torch.randn(3, 8, 32, device="cuda")[:, :5])
    with pytest.raises(ValueError, match="w must hold"):
        etpc.etpc_layer_norm(x, torch.ones(31, device="cuda"))
    with pytest.raises(TypeError):
        etpc.etpc_layer_norm(x, torch.ones(32, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="shape"):
        etpc.etpc_layer_norm_backward(x, x[:5], mean, rstd)
    with pytest.raises(TypeError):
        etpc.etpc_layer_norm_backward(x, x.bfloat16(), mean, rstd)
    with pytest.raises(ValueError, match="mean"):
        etpc.etpc_layer_norm_backward(x, x, mean[:5], rstd)
    with pytest.raises(etpc.EtpcError, match="overlap"):
        etpc.etpc_layer_norm(x, y=x)
    with pytest.raises(etpc.EtpcError, match="probability"):
        etpc.etpc_dropout(x, 1.5, 0)
    with pytest.raises(ValueError, match="offset"):
        etpc.etpc_dropout(x, 0.5, 0, torch.zeros(1, device="cuda"))
    with pytest.raises(etpc.EtpcError, match="small"):
        big = torch.randn(5000, 64, device="cuda")
        m = torch.ones(5000, device="cuda")
        etpc.etpc_layer_norm_backward(big, big.clone(), m, m, ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="stats"):
        etpc.etpc_irreps_norm_backward("8x0e+8x1o", x, x.clone(), torch.ones(6, 2, device="cuda"))
