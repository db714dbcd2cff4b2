"""Feed-forward operators where they can go wrong: NaN and infinities, memory beside the results, repeated rows,
streams, captured graphs, subsets of the results, addresses past 32 bits."""
import math

import numpy as np
import pytest
import torch

from oracle import feedforward as ff
from tests.gpu_helpers import note
from tests.test_gpu_linear import DTYPES, KINDS, check_backward, check_forward, f64, matrix, vector, weights

pytestmark = pytest.mark.gpu

# rows, inputs, outputs: every path of the layer (one or two rows, narrow rows, tiles by one, tiles in ranges of k, large tiles)
PATHS = ((1, 300, 200), (2, 72, 264), (40, 64, 64), (40, 8, 96), (70, 264, 200), (20, 3000, 136), (20, 3001, 135), (3000, 264, 264),
         (2100, 136, 2056))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _etpc():
    import equivariant_gnn_tensor_amd as etpc
    return etpc


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("act", ff.ACTS)
def test_activations_of_not_finite_numbers(kind, act):
    """z is the bias where x is zero: limits of the activations and their slopes, NaN kept."""
    etpc = _etpc()
    special = torch.tensor([math.inf, -math.inf, math.nan, 0.0, -0.0, 1.0], device="cuda")
    want = {"none": special, "relu": special.clamp(min=0), "silu": torch.tensor([math.inf, 0, math.nan, 0, 0, 0.7310586]).cuda(),
            "gelu": torch.tensor([math.inf, 0, math.nan, 0, 0, 0.8413447]).cuda(), "tanh": torch.tanh(special)}[act]
    slopes = {"none": [1] * 6, "relu": [1, 0, math.nan, 0, 0, 1], "silu": [1, 0, math.nan, 0.5, 0.5, 0.9276706],
              "gelu": [1, 0, math.nan, 0.5, 0.5, 1.0833155], "tanh": [0, 0, math.nan, 1, 1, 0.4199743]}[act]
    tol = {"f32": 1e-6, "bf16": 2.0 ** -7, "f16": 2.0 ** -10}[kind]   # two half steps
    for rows, n_in, n_out in PATHS:
        note(f"special numbers {kind} {act} {rows}x{n_in}->{n_out}")
        x, w = torch.zeros(rows, n_in, dtype=DTYPES[kind], device="cuda"), torch.zeros(n_in, n_out, dtype=DTYPES[kind], device="cuda")
        b = special.repeat(n_out)[:n_out].contiguous()
        y, z = etpc.etpc_linear(x, w, b, act=act)
        ref = want.repeat(n_out)[:n_out].expand(rows, n_out)
        assert torch.allclose(y.float(), ref.float(), rtol=tol, atol=tol, equal_nan=True)
        if z is not None:
            assert torch.equal(z.float().nan_to_num(7), b.expand(rows, n_out).nan_to_num(7))
            y_bar = torch.ones_like(y)
            _, _, b_bar = etpc.etpc_linear_backward(x, w, y_bar, z=z, act=act)
            s = rows * torch.tensor(slopes, device="cuda").repeat(n_out)[:n_out]
            assert torch.allclose(b_bar, s, rtol=1e-4, equal_nan=True)


@pytest.mark.parametrize("kind", KINDS)
def test_not_finite_rows_stay_apart(kind):
    """A NaN or infinity in x or y_bar reaches its own row (and the weights' gradient) only."""
    etpc = _etpc()
    rng = np.random.default_rng(4)
    for rows, n_in, n_out in PATHS:
        if rows < 2:
            continue
        x, w, b = matrix(rng, rows, n_in, kind), weights(rng, n_in, n_out, kind, "io"), vector(rng, n_out)
        y_bar = matrix(rng, rows, n_out, kind)
        good = etpc.etpc_linear(x, w, b)[0], etpc.etpc_linear_backward(x, w, y_bar, want=("x",))[0]
        x2, y2 = x.clone(), y_bar.clone()
        x2[1, n_in // 2], y2[1, n_out - 1] = math.nan, math.inf
        bad = etpc.etpc_linear(x2, w, b)[0], etpc.etpc_linear_backward(x, w, y2, want=("x",))[0]
        for g, h in zip(good, bad):
            keep = [k for k in range(rows) if k != 1]
            assert torch.equal(g[keep], h[keep]) and not torch.isfinite(h[1]).any()


@pytest.mark.parametrize("kind", KINDS)
def test_memory_beside_the_results(kind):
    etpc = _etpc()
    rng = np.random.default_rng(6)

    def canvas(n, cols, dtype):
        full = torch.full((n + 2, cols + 9), 7.0, dtype=dtype, device="cuda")
        return full, full[1:n + 1, 3:cols + 3]

    def untouched(full, view):
        copy = full.clone()
        copy[1:view.shape[0] + 1, 3:view.shape[1] + 3] = 7.0
        return bool((copy == 7.0).all())
    for rows, n_in, n_out in PATHS:
        dt = DTYPES[kind]
        x, w, b = matrix(rng, rows, n_in, kind, 5), weights(rng, n_in, n_out, kind, "oi", 3), vector(rng, n_out)
        res, y_bar = matrix(rng, rows, n_out, kind, 1), matrix(rng, rows, n_out, kind, 2)
        (fy, y), (fz, z), (fx, xb), (fw, wb) = (canvas(rows, n_out, dt), canvas(rows, n_out, dt), canvas(rows, n_in, dt),
                                               canvas(n_out, n_in, dt))
        etpc.etpc_linear(x, w, b, residual=res, act="silu", y=y, z=z)
        check_forward(y, z, f64(x), f64(w), f64(b), f64(res), "silu", kind)
        bb = torch.full((n_out + 2,), 7.0, device="cuda")
        etpc.etpc_linear_backward(x, w, y_bar, z=z, act="silu", outs=(xb, wb.t(), bb[1:-1]))
        check_backward(xb, wb.t(), bb[1:-1], f64(x), f64(w), f64(y_bar), f64(z), "silu", kind)
        assert untouched(fy, y) and untouched(fz, z) and untouched(fx, xb) and untouched(fw, wb)
        assert float(bb[0]) == 7.0 and float(bb[-1]) == 7.0
    for n, cols in ((1, 5), (3, 64), (70, 577), (40, 1032), (5, 8200)):
        x = matrix(rng, n, cols, kind, 4)
        (fy, y), (fh, h), (fg, gb), (fr, rb), (fx, xb) = (canvas(n, cols, DTYPES[kind]) for _ in range(5))
        _, _, stats = etpc.etpc_norm_gate_add_norm(x, gate=x, residual=x, y=y, h=h)
        etpc.etpc_norm_gate_add_norm_backward(x, h, x, stats, gate=x, outs=(xb, gb, rb) + (None,) * 5)
        ref = etpc.etpc_norm_gate_add_norm(x, gate=x, residual=x)
        bars = etpc.etpc_norm_gate_add_norm_backward(x, ref[1], x, ref[2], gate=x)
        for a, b in zip((y, h, xb, gb, rb), (ref[0], ref[1], *bars[:3])):
            assert torch.equal(a, b)
        assert all(untouched(f, v) for f, v in ((fy, y), (fh, h), (fg, gb), (fr, rb), (fx, xb)))


@pytest.mark.parametrize("kind", KINDS)
def test_repeated_rows(kind):
    """One row for all (stride 0) equals the same rows written out."""
    etpc = _etpc()
    rng = np.random.default_rng(7)
    for rows, n_in, n_out in PATHS:
        w, b = weights(rng, n_in, n_out, kind, "io"), vector(rng, n_out)
        x, y_bar = (matrix(rng, 1, n, kind).expand(rows, n) for n in (n_in, n_out))
        for args in ((x, y_bar), (x.contiguous(), y_bar.contiguous())):
            y, z = etpc.etpc_linear(args[0], w, b, residual=args[1], act="gelu")
            check_forward(y, z, f64(x), f64(w), f64(b), f64(y_bar), "gelu", kind)
            bars = etpc.etpc_linear_backward(args[0], w, args[1], z=z, act="gelu")
            check_backward(*bars, f64(x), f64(w), f64(y_bar), f64(z), "gelu", kind)
    g = matrix(rng, 1, 200, kind).expand(33, 200)
    x, yb = matrix(rng, 33, 200, kind), matrix(rng, 33, 200, kind)
    out = [etpc.etpc_norm_gate_add_norm(x, gate=t, residual=t) for t in (g, g.contiguous())]
    assert all(torch.equal(a, b) for a, b in zip(*out))
    bars = [etpc.etpc_norm_gate_add_norm_backward(x, out[0][1], yb, out[0][2], gate=t) for t in (g, g.contiguous())]
    assert bars[0][1].shape == (33, 200) and all(torch.equal(a, b) for a, b in zip(*bars))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_subsets_axes_and_repetition(kind):
    """Each result on its own, given leading axes, and a second run: the same bits."""
    etpc = _etpc()
    rng = np.random.default_rng(8)
    for rows, n_in, n_out in PATHS:
        x, w, b = matrix(rng, rows, n_in, kind), weights(rng, n_in, n_out, kind, "oi"), vector(rng, n_out)
        y_bar = matrix(rng, rows, n_out, kind)
        y, z = etpc.etpc_linear(x, w, b, act="silu")
        assert torch.equal(y, etpc.etpc_linear(x, w, b, act="silu", keep_z=False)[0])
        whole = etpc.etpc_linear_backward(x, w, y_bar, z=z, act="silu")
        again = etpc.etpc_linear_backward(x, w, y_bar, z=z, act="silu")
        assert all(torch.equal(p, q) for p, q in zip(whole, again))
        for k, name in enumerate("xwb"):
            only = etpc.etpc_linear_backward(x, w, y_bar, z=z, act="silu", want=(name,))
            assert torch.equal(only[k], whole[k]) and all(only[j] is None for j in range(3) if j != k)
        if rows % 2 == 0:
            y3, z3 = etpc.etpc_linear(x.view(2, rows // 2, n_in), w, b, act="silu")
            assert y3.shape == (2, rows // 2, n_out) and torch.equal(y3.view(rows, n_out), y)
    x, yb = matrix(rng, 300, 264, kind), matrix(rng, 300, 264, kind)
    y, h, stats = etpc.etpc_norm_gate_add_norm(x, gate=yb, residual=x)
    names = ("x", "gate", "residual", "w1", "b1", "scale", "w2", "b2")
    whole = etpc.etpc_norm_gate_add_norm_backward(x, h, yb, stats, gate=yb, h_bar=x)
    for k, name in enumerate(names):
        only = etpc.etpc_norm_gate_add_norm_backward(x, h, yb, stats, gate=yb, h_bar=x, want=(name,))
        assert torch.equal(only[k], whole[k]) and sum(t is not None for t in only) == 1
    assert torch.equal(y, etpc.etpc_norm_gate_add_norm(x, gate=yb, residual=x, keep_h=False, keep_stats=False)[0])


def _block_step(etpc, p, x, t):
    """Two layers around the gated join, their gradients, and clipping: the operators as they follow one another."""
    u, zu = etpc.etpc_linear(x, p["A"], p["a"], act="gelu")
    v, _ = etpc.etpc_linear(u, p["B"])
    y, h, stats = etpc.etpc_norm_gate_add_norm(v, gate=t, residual=x, w1=p["w1"])
    v_bar, g_bar, _, w1_bar, *_ = etpc.etpc_norm_gate_add_norm_backward(v, h, t, stats, gate=t, w1=p["w1"])
    u_bar, B_bar, _ = etpc.etpc_linear_backward(u, p["B"], v_bar, want=("x", "w"))
    x_bar, A_bar, a_bar = etpc.etpc_linear_backward(x, p["A"], u_bar, z=zu, act="gelu")
    grads = [A_bar, a_bar, B_bar, w1_bar]
    outs = [torch.empty_like(g) for g in grads]
    norm = etpc.etpc_clip_grad_norm(grads, 0.5, outs=outs)
    return [y, h, stats, g_bar, x_bar, norm, *outs]


def _block_data(kind, rows, c, hidden):
    rng = np.random.default_rng(9)
    p = dict(A=weights(rng, c, hidden, kind, "io"), a=vector(rng, hidden), B=weights(rng, hidden, c, kind, "oi"), w1=vector(rng, c))
    return p, [matrix(rng, rows, c, kind) for _ in range(3)], [matrix(rng, rows, c, kind) for _ in range(3)]


@pytest.mark.parametrize("kind,rows,c,hidden", [("f32", 200, 64, 128), ("bf16", 700, 264, 1032), ("f16", 33, 520, 2056), ("bf16", 2, 64, 96)])
def test_captured_and_on_another_stream(kind, rows, c, hidden):
    """The sequence captured into a graph, replayed on other inputs with eager work between, and on a side stream:
    the eager results' bits each time."""
    etpc = _etpc()
    p, xs, ts = _block_data(kind, rows, c, hidden)
    want = [[r.clone() for r in _block_step(etpc, p, x, t)] for x, t in zip(xs, ts)]
    x, t = xs[0].clone(), ts[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for k in range(3):
            got = _block_step(etpc, p, xs[k], ts[k])
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want[k]))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _block_step(etpc, p, x, t)
    for k in (0, 1, 2, 1):
        x.copy_(xs[k])
        t.copy_(ts[k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[k])), k
        assert all(torch.equal(a, b) for a, b in zip(_block_step(etpc, p, xs[k], ts[k]), want[k]))


def test_explicit_stream_and_workspace():
    """A stream given as an argument, and one workspace for call after call."""
    etpc = _etpc()
    rng = np.random.default_rng(10)
    x, w, y_bar = matrix(rng, 700, 264, "bf16"), weights(rng, 264, 520, "bf16", "io"), matrix(rng, 700, 520, "bf16")
    want = etpc.etpc_linear_backward(x, w, y_bar)
    ws = torch.empty(etpc.etpc_linear_backward_workspace_size(700, 264, 520, torch.bfloat16), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = etpc.etpc_linear_backward(x, w, y_bar, ws=ws, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    few, long = matrix(rng, 20, 3000, "bf16"), weights(rng, 3000, 136, "bf16", "oi")
    ws = torch.empty(etpc.etpc_linear_workspace_size(20, 3000, 136, torch.bfloat16), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    assert torch.equal(etpc.etpc_linear(few, long, ws=ws)[0], etpc.etpc_linear(few, long)[0])
    with pytest.raises(etpc.EtpcError, match="WORKSPACE|workspace"):
        etpc.etpc_linear(few, long, ws=ws[:64])


def test_refusals_on_the_device():
    etpc = _etpc()
    x, w = torch.zeros(4, 8, device="cuda"), torch.zeros(8, 16, device="cuda")
    for call, error, word in (
            (lambda: etpc.etpc_linear(x, w.bfloat16()), TypeError, "float32"), (lambda: etpc.etpc_linear(x, w[:7]), ValueError, "inputs"),
            (lambda: etpc.etpc_linear(x, w, torch.zeros(15, device="cuda")), ValueError, "16 numbers"),
            (lambda: etpc.etpc_linear(x, torch.zeros(8, 32, device="cuda")[:, ::2]), ValueError, "contiguous"),
            (lambda: etpc.etpc_linear(x, w.cpu()), ValueError, "expected"), (lambda: etpc.etpc_linear(x, w, y=x), ValueError, "shape"),
            (lambda: etpc.etpc_linear_backward(x, w, torch.zeros(4, 16, device="cuda"), act="silu"), ValueError, "needs z"),
            (lambda: etpc.etpc_norm_gate_add_norm(x, gate=x[:3]), ValueError, "gate"),
            (lambda: etpc.etpc_norm_gate_add_norm(x, y=x), etpc.EtpcError, "overlap"),
            (lambda: etpc.etpc_clip_grad_norm([x, x], 1.0), etpc.EtpcError, "overlap"),
            (lambda: etpc.etpc_clip_grad_norm([x], 1.0, outs=[w]), ValueError, "like its tensor"),
            (lambda: etpc.etpc_grad_norm([x, w.cpu()]), ValueError, "GPU")):
        with pytest.raises(error, match=word):
            call()


def test_offsets_past_32_bits():
    """Results, partial sums and tensors of more than 2^32 bytes: the last rows and elements are right."""
    etpc = _etpc()
    rng = np.random.default_rng(12)
    rows, n_in, n_out = 540000, 8, 4096
    w, b = weights(rng, n_in, n_out, "bf16", "io"), vector(rng, n_out)
    tail = matrix(rng, 300, n_in, "bf16")
    x = torch.zeros(rows, n_in, dtype=torch.bfloat16, device="cuda")
    x[-300:] = tail
    note("layer with 4.4 GB of results")
    y, _ = etpc.etpc_linear(x, w, b)
    assert y.numel() * 2 > 1 << 32
    assert torch.equal(y[-300:], etpc.etpc_linear(x[-300:], w, b)[0]) and torch.equal(y[0], b.bfloat16())
    note("its gradient")
    x_bar, _, _ = etpc.etpc_linear_backward(x, w, y, want=("x",))
    assert torch.equal(x_bar[-300:], etpc.etpc_linear_backward(x[-300:], w, y[-300:].contiguous(), want=("x",))[0])
    note("gated join over the same rows")
    out, h, stats = etpc.etpc_norm_gate_add_norm(y, residual=y)
    few = etpc.etpc_norm_gate_add_norm(y[-300:], residual=y[-300:])
    assert torch.equal(out[-300:], few[0]) and torch.equal(h[-300:], few[1]) and torch.equal(stats[-300:], few[2])
    del out, h, y
    note("one row of 33 million results")
    n = (1 << 25) + 5
    w = torch.randn(1, n, device="cuda").bfloat16()
    for v in (w, w.t().contiguous().t()):   # both layouts of [1, n] weights
        y, _ = etpc.etpc_linear(torch.full((1, 1), 2.0, dtype=torch.bfloat16, device="cuda"), v)
        assert torch.equal(y, 2 * w)
    note("norm of 4.3 GB")
    g = torch.zeros((1 << 31) + 5, dtype=torch.bfloat16, device="cuda")
    g[-1], g[0] = 4.0, 3.0
    assert float(etpc.etpc_clip_grad_norm([g], 2.5)) == 5.0
    assert float(g[-1]) == 2.0 and float(g[0]) == 1.5


def test_most_rows():
    """2^31 - 1 rows: tile numbers and ends of the ranges of rows within their types (x and y_bar are one row for all)."""
    etpc = _etpc()
    rows = (1 << 31) - 1
    rng = np.random.default_rng(14)
    note("layer of 2^31 - 1 rows to one output")
    one, w = matrix(rng, 1, 200, "bf16"), weights(rng, 200, 1, "bf16", "io")
    y, _ = etpc.etpc_linear(one.expand(rows, 200), w)
    few = etpc.etpc_linear(one.expand(3, 200), w)[0]
    assert bool((y == y[0]).all())
    check_forward(y[-3:], None, f64(one.expand(3, 200)), f64(w), np.zeros(1), None, "none", "bf16")
    assert torch.equal(y[:3], y[-3:]) and y.shape == (rows, 1) and few.shape == (3, 1)
    del y
    note("weight gradient over 2^31 - 1 rows")
    x = torch.ones(1, 130, dtype=torch.bfloat16, device="cuda").expand(rows, 130)
    y_bar = torch.ones(1, 1, dtype=torch.bfloat16, device="cuda").expand(rows, 1)
    w = torch.ones(130, 1, dtype=torch.bfloat16, device="cuda")
    _, w_bar, b_bar = etpc.etpc_linear_backward(x, w, y_bar, want=("w", "b"))
    # whole numbers up to 2^24 in a range are exact; the sums of up to 1024 ranges round once each
    assert float((w_bar.double() / rows - 1).abs().max()) <= 2.0 ** -8 + 1024 * 2.0 ** -24
    assert abs(float(b_bar) / rows - 1) <= 1024 * 2.0 ** -24
