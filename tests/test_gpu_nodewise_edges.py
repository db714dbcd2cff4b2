"""GPU checks of the node-wise operators where they can go wrong, against oracle/nodewise.py
(float64): rows that hold a NaN or an infinity, the stored mean of rows near zero, rows of
2^25 and more columns, single rows between the columns of others, outputs left out.

`same` compares values that are not finite by kind: NaN with NaN, an infinity with the
infinity of its sign.  u = 2^-24.
"""
import numpy as np
import pytest
import torch

from oracle import nodewise as nw
from tests.gpu_helpers import note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5


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


def same(got, ref, bound, what):
    """Equal where ref is not finite, within bound elsewhere."""
    got, bound = f64(got), np.broadcast_to(bound, ref.shape)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), (what, np.argwhere(np.isnan(got) != np.isnan(ref))[:4])
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), what
    ok = np.isfinite(ref)
    bad = ~(np.abs(got[ok] - ref[ok]) <= bound[ok])
    assert not bad.any(), (what, got[ok][bad][:4], ref[ok][bad][:4], bound[ok][bad][:4])


# ---------------------------------------------------------------- NaN and infinities

@pytest.mark.parametrize("cols", [5, 64, 600, 3000, 18000])
@pytest.mark.parametrize("join", [False, True])
def test_a_nan_in_a_row_reaches_its_statistics(cols, join):
    """A row with a NaN has neither mean nor rstd, one with an infinity has an infinite mean and
    no rstd; neither has a finite y, and no other row is touched."""
    etpc = _etpc()
    rng = np.random.default_rng(cols)
    clean = rng.standard_normal((9, cols)).astype(np.float32)
    bad = clean.copy()
    bad[2, cols // 2], bad[5, 0], bad[7, cols - 1] = np.nan, np.inf, -np.inf
    note(f"layer norm of rows with NaN, cols={cols} join={join}")

    def forward(a):
        x = tensor(a)
        if not join:
            return etpc.etpc_layer_norm(x, eps=EPS)
        y, h, mean, rstd = etpc.etpc_dropout_add_layer_norm(x, torch.zeros_like(x), eps=EPS)
        assert torch.equal(h.nan_to_num(1.5), x.nan_to_num(1.5))
        return y, mean, rstd

    good, got = forward(clean), forward(bad)
    keep = torch.tensor([0, 1, 3, 4, 6, 8], device="cuda")
    for p, q in zip(good, got):
        assert torch.equal(p[keep], q[keep])
    y, mean, rstd = got
    assert torch.isnan(mean[2]) and torch.isnan(rstd[[2, 5, 7]]).all() and torch.isnan(y[[2, 5, 7]]).all()
    assert mean[5] == float("inf") and mean[7] == -float("inf")


# flat segments (narrow or l = 0), channel by channel, more channels than a wave keeps
@pytest.mark.parametrize("text", ["8x0e+8x1o", "5x1o+3x2e+2x3o+9x0e", "64x0e+64x1o+64x2e+64x3o", "26x1o+33x2e+45x3o",
                                  "300x1o+258x2e", "700x3o+2100x0e+600x1e"])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_a_nan_in_an_irreps_block_spoils_the_block(text, value):
    """One value of one block of one node: the block's y and statistics are what the definition
    makes of it (NaN everywhere for a NaN), all other blocks and nodes keep their bits."""
    etpc = _etpc()
    ir, d = etpc.parse_irreps(text), etpc.etpc_irreps_dims(text)
    rng = np.random.default_rng(d["dim"])
    n = 11
    clean = rng.standard_normal((n, d["dim"])).astype(np.float32)
    w, b = tensor(rng.standard_normal(d["channels"])), tensor(rng.standard_normal(d["biases"]))
    y0, s0 = etpc.etpc_irreps_norm(text, tensor(clean), w, b, eps=EPS)
    for k, (mul, l, _, off, ch, _) in enumerate(nw.blocks(ir)):
        note(f"irreps norm {text} with {value} in block {k}")
        width, bad = mul * (2 * l + 1), clean.copy()
        bad[4, off + width // 2] = value
        y, stats = etpc.etpc_irreps_norm(text, tensor(bad), w, b, eps=EPS)
        with np.errstate(invalid="ignore"):
            ry, rs = nw.irreps_norm(bad, ir, f64(w), f64(b), EPS)
        part = slice(off, off + width)
        same(y[4, part], ry[4, part], 256 * U * np.abs(ry[4, part]), (text, k, "y"))
        same(stats[4, k], rs[4, k], 0.0, (text, k, "stats"))   # none of them finite but 0
        other = torch.ones_like(y, dtype=torch.bool)
        other[4, part] = False
        assert torch.equal(y[other], y0[other])
        other = torch.ones_like(stats, dtype=torch.bool)
        other[4, k] = False
        assert torch.equal(stats[other], s0[other])
        if np.isnan(value):   # the gradients' sums show it too
            _, wb, _ = etpc.etpc_irreps_norm_backward(text, tensor(bad), y0, stats, w)
            assert torch.isnan(wb[ch:ch + mul]).all() and torch.isfinite(wb[:ch]).all() and torch.isfinite(wb[ch + mul:]).all()


# ---------------------------------------------------------------- the stored mean

@pytest.mark.parametrize("cols", [20, 100, 600, 1000, 3000, 12000, 18000])
@pytest.mark.parametrize("level", [0, 1, 37, 1000])
def test_stored_mean_of_rows_near_zero(cols, level):
    """Pairs a, -a of numbers in [1, 2) on a grid of 2^-18, `level` steps of which are added to
    the first 2/3 of the row: every partial sum is a multiple of 2^-18 below 2^6, hence exact
    in 24 bits, and the stored mean is off by the roundings of its division and of what may
    still be added to it, 2 u of itself.  (The differences x - mean are not exact: their
    average is off by up to half a step of [1, 2), 2^-24, which is 1e-2 of these means.)"""
    etpc = _etpc()
    rng = np.random.default_rng(cols + level)
    step = 2.0 ** -18
    a = 1.0 + rng.integers(2000, (1 << 18) - 2000, (6, cols // 2)) * step
    a *= rng.choice([-1.0, 1.0], a.shape)
    x = np.stack([a, -a], axis=-1).reshape(6, cols)
    x[:, :2 * cols // 3] += level * step
    assert 2 + cols * level * step < 128 and x.sum(axis=1).max() < 64 and np.array_equal(x, x.astype(np.float32))
    note(f"stored mean near zero, cols={cols} level={level}")
    ref, t = x.mean(axis=1), tensor(x)
    yb = tensor(np.zeros((6, cols)))
    means = [etpc.etpc_layer_norm(t, eps=EPS)[1], etpc.etpc_dropout_add_layer_norm(t, yb, eps=EPS)[2],
             etpc.etpc_irreps_norm(f"{cols}x0e", t, eps=EPS)[1][:, 0, 0]]
    for m in means:
        same(m, ref, 2 * U * np.abs(ref), "mean")


# ---------------------------------------------------------------- very long rows

@pytest.mark.parametrize("kind,cols", [(torch.bfloat16, (1 << 25) + 3), (torch.float32, 1 << 26)])
def test_gradients_of_rows_past_2_to_the_25(kind, cols):
    """Both stages of the parameter gradients' sums at row lengths where the second stage's
    columns, sixteen a workgroup of 1024 threads, are more than one launch holds.  Two rows:
    one difference, two products and one sum, 5 u of their magnitudes."""
    etpc = _etpc()
    torch.manual_seed(3)
    x, yb = torch.randn(2, cols, device="cuda").to(kind), torch.randn(2, cols, device="cuda").to(kind)
    mean, rstd = torch.tensor([0.25, -0.5], device="cuda"), torch.tensor([1.5, 0.75], device="cuda")
    note(f"parameter gradients of rows of {cols} columns")
    x_bar, wb, bb = etpc.etpc_layer_norm_backward(x, yb, mean, rstd, want=("w", "b"))
    assert x_bar is None and wb.shape == bb.shape == (cols,)
    t = yb.double() * (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    assert ((wb.double() - t.sum(0)).abs() <= 5 * U * t.abs().sum(0)).all()
    t = yb.double()
    assert ((bb.double() - t.sum(0)).abs() <= U * t.abs().sum(0)).all()


# ---------------------------------------------------------------- where operands may lie

def test_a_broadcast_row_between_the_columns_of_the_output():
    """One row read for all rows may lie in the gap between two rows of the output: their
    extents cross, their numbers do not.  One that meets a row is refused."""
    etpc = _etpc()
    rng = np.random.default_rng(2)
    big = tensor(rng.standard_normal((23, 150)))
    before = big.clone()
    for r in (0, 7, 22):
        big.copy_(before)
        res, y = big[r:r + 1, 64:128].expand(23, 64), big[:, :64]
        x = tensor(rng.standard_normal((23, 64)))
        note(f"broadcast row {r} between the rows of y")
        got = etpc.etpc_dropout_add_layer_norm(x, res, y=y, eps=EPS)
        ref = etpc.etpc_dropout_add_layer_norm(x, res.contiguous(), eps=EPS)
        assert got[0] is y and torch.equal(y, ref[0]) and torch.equal(got[1], ref[1])
        assert torch.equal(big[:, 64:], before[:, 64:])
        for meets in (big[r:r + 1, 63:127], big[r:r + 1, 0:64]):
            with pytest.raises(etpc.EtpcError, match="overlap"):
                etpc.etpc_dropout_add_layer_norm(x, meets.expand(23, 64), y=y, eps=EPS)
    last = big.view(-1)[86:150]   # the gap before row 1: ends where the row starts
    etpc.etpc_layer_norm(last.expand(23, 64), y=big[:, :64])
    with pytest.raises(etpc.EtpcError, match="overlap"):
        etpc.etpc_layer_norm(big.view(-1)[87:151].expand(23, 64), y=big[:, :64])


def test_statistics_in_the_gaps_of_feature_rows():
    """Statistics and parameter gradients as parts of one buffer, and in the columns that a
    strided matrix leaves free, are apart from it and from one another."""
    etpc = _etpc()
    rng = np.random.default_rng(4)
    n, cols = 12, 40
    x, yb = tensor(rng.standard_normal((n, cols))), tensor(rng.standard_normal((n, cols)))
    w = tensor(rng.standard_normal(cols))
    ref = etpc.etpc_layer_norm(x, w, eps=EPS)
    big = torch.zeros(n, 80, device="cuda")
    note("statistics beside y")
    got = etpc.etpc_layer_norm(x, w, y=big[:, :cols], mean=big[3, 40:52], rstd=big[11, 68:80], eps=EPS)
    assert all(torch.equal(p, q) for p, q in zip(got, ref))
    _, wb, bb = etpc.etpc_layer_norm_backward(x, yb, ref[1], ref[2], w)
    flat = torch.zeros(2 * cols, device="cuda")
    outs = (big[:, 40:], flat[:cols], flat[cols:])
    etpc.etpc_layer_norm_backward(x, yb, ref[1], ref[2], w, outs=outs)
    assert torch.equal(outs[1], wb) and torch.equal(outs[2], bb)
    with pytest.raises(etpc.EtpcError, match="overlap"):
        etpc.etpc_layer_norm_backward(x, yb, ref[1], ref[2], w, outs=(None, flat[:cols], flat[cols - 1:-1]))


# ---------------------------------------------------------------- outputs left out

@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("cols", [7, 64, 577, 2048, 18000])
def test_join_without_its_sum(kind, cols):
    """keep_h=False (a forward pass with no backward) leaves h out and changes nothing else."""
    etpc = _etpc()
    torch.manual_seed(cols)
    x, res = torch.randn(37, cols, device="cuda").to(kind), torch.randn(37, cols, device="cuda").to(kind)
    w = torch.randn(cols, device="cuda")
    note(f"join without h, {kind} cols={cols}")
    for p in (0.0, 0.3):
        y, h, mean, rstd = etpc.etpc_dropout_add_layer_norm(x, res, w, p=p, seed=3, offset=4)
        got = etpc.etpc_dropout_add_layer_norm(x, res, w, p=p, seed=3, offset=4, keep_h=False)
        assert got[1] is None and torch.equal(got[0], y) and torch.equal(got[2], mean) and torch.equal(got[3], rstd)
        got = etpc.etpc_dropout_add_layer_norm(x, res, w, p=p, seed=3, offset=4, keep_h=False, stats=False)
        assert got[1:] == (None, None, None) and torch.equal(got[0], y)
        given = torch.empty_like(x)   # a given h is written all the same
        got = etpc.etpc_dropout_add_layer_norm(x, res, w, p=p, seed=3, offset=4, h=given, keep_h=False)
        assert got[1] is given and torch.equal(given, h)
