"""Timed cases of the node-wise operators: layer norm, dropout, their residual join, irreps norm.

Each case runs one operator in one direction.  `own = False` computes it with elementary
torch operations in 32 bits; `own = True` calls this package.  `exact` gives the same
outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5
# The hidden features of the bundled workloads: 64 atoms; 4096 atoms and batches of cells; 16384 atoms channelwise.
IRREPS_TINY = "8x0e+8x1o"
IRREPS_MACE = "64x0e+64x1o+64x2e"
IRREPS_MACE_OUT = "64x0e+64x1o+64x2e+64x3o"
IRREPS_CHANNEL = "128x0e+128x1o+128x2e+128x3o"


def listed():
    return [
        # one row of invariants through a readout's norm at inference: latency
        dict(name="norm_one_row", op="norm", dir="fwd", dtype="f32", rows=1, cols=1024, pitch=1024),
        # the scalar block inside wide feature rows of a batch of 511 cells: strided input
        dict(name="norm_scalar_block", op="norm", dir="fwd", dtype="f32", rows=65408, cols=64, pitch=576),
        # hidden rows of a radial network on the 214980 edges of the 4096-atom graph, training
        dict(name="norm_edges_bwd", op="norm", dir="bwd", dtype="bf16", rows=214980, cols=64, pitch=64),
        # wide invariant rows, training in half precision
        dict(name="norm_wide_bwd", op="norm", dir="bwd", dtype="f16", rows=8192, cols=4096, pitch=4096),
        # a small batch's invariants: latency
        dict(name="dropout_small", op="dropout", dir="fwd", dtype="f32", rows=64, cols=64, pitch=64, p=0.1),
        # invariants of 511 cells of 128 atoms: throughput (the backward is the same call on the gradient)
        dict(name="dropout_large", op="dropout", dir="fwd", dtype="bf16", rows=65408, cols=1024, pitch=1024, p=0.1),
        # equivariant features of 16384 atoms: a channel's components live or die together
        dict(name="dropout_irreps", op="irreps_dropout", dir="fwd", irreps=IRREPS_CHANNEL, rows=16384, p=0.2),
        # residual block on the invariants of 511 cells, forward in training
        dict(name="join_large_fwd", op="join", dir="fwd", dtype="bf16", rows=65408, cols=1024, p=0.1),
        # the same block's gradient at odd sizes
        dict(name="join_odd_bwd", op="join", dir="bwd", dtype="f32", rows=4097, cols=2047, p=0.15),
        # tiny graph: latency of a training step's backward
        dict(name="irreps_norm_tiny_bwd", op="irreps_norm", dir="bwd", irreps=IRREPS_TINY, rows=64),
        # features between two convolutions of the 4096-atom graph
        dict(name="irreps_norm_fwd", op="irreps_norm", dir="fwd", irreps=IRREPS_MACE_OUT, rows=4096),
        # the gradient for a batch of 511 cells
        dict(name="irreps_norm_large_bwd", op="irreps_norm", dir="bwd", irreps=IRREPS_MACE, rows=65408),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "dropout", "irreps_dropout", "join", "irreps_norm", "irreps_norm"])
    if op.startswith("irreps"):
        blocks, dim = [], 0
        for _ in range(rng.randint(1, 6)):
            l, mul = rng.randint(0, 3), _log(rng, 4, 256)
            if rng.random() < 0.6:   # multiples of eight are usual, others occur
                mul = max(8, mul // 8 * 8)
            blocks.append("%dx%d%s" % (mul, l, rng.choice("eo")))
            dim += mul * (2 * l + 1)
        case = dict(op=op, dir="fwd", irreps="+".join(blocks), rows=_log(rng, 1, min(1 << 17, (1 << 25) // dim)))
        if op == "irreps_norm":
            case["dir"] = rng.choice(["fwd", "bwd"])
        else:
            case["p"] = round(rng.uniform(0.02, 0.6), 3)
        return case
    cols = _log(rng, 1 if op == "dropout" else 4, 16384)
    if rng.random() < 0.5 and cols > 16:
        cols = cols // 16 * 16
    rows = _log(rng, 1, min(1 << 18, (1 << (24 if op == "join" else 25)) // cols))
    case = dict(op=op, dir=rng.choice(["fwd", "bwd"]) if op != "dropout" else "fwd", dtype=rng.choice(["f32", "bf16", "f16"]), rows=rows,
                cols=cols)
    if op != "join":
        case["pitch"] = cols + rng.choice([0, 0, 0, 8, 5])
    if op != "norm":
        case["p"] = round(rng.uniform(0.02, 0.6), 3)
    return case


def _irreps(text):
    """[(multiplicity, degree, parity, offset in a row, offset among channels)], row width, channels, 0e channels."""
    blocks, dim, channels, biases = [], 0, 0, 0
    for token in text.split("+"):
        mul, ir = token.split("x")
        mul, l = int(mul), int(ir[0])
        blocks.append((mul, l, ir[1], dim, channels))
        dim += mul * (2 * l + 1)
        channels += mul
        biases += mul if ir == "0e" else 0
    return blocks, dim, channels, biases


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = dict(case=case, rng_seed=(seed * 0x9E3779B97F4A7C15 + 12345) % (1 << 64), rng_offset=(seed * 7919 + 3) % (1 << 40))
    rows, op = case["rows"], case["op"]
    if op.startswith("irreps"):
        s["irreps"] = _irreps(case["irreps"])
        blocks, dim, channels, biases = s["irreps"]
        s["x"] = normal(rows, dim) * (0.5 + torch.rand(rows, 1, generator=gen, device="cuda"))
        if op == "irreps_norm":
            s["w"], s["b"] = 1.0 + 0.1 * normal(channels), 0.1 * normal(biases)
            if case["dir"] == "bwd":
                s["stats"] = _irreps_stats(s["x"], blocks)
                s["y_bar"] = 0.1 * normal(rows, dim)
        return s
    cols, dtype = case["cols"], DTYPES[case["dtype"]]
    channel = 0.3 * normal(cols)   # channels have levels of their own

    def features(pitch=cols):
        full = torch.empty(rows, pitch, device="cuda", dtype=dtype).fill_(0.25)
        full[:, :cols] = ((normal(rows, cols) + channel) * (0.5 + torch.rand(rows, 1, generator=gen, device="cuda"))).to(dtype)
        return full[:, :cols]

    s["x"] = features(case.get("pitch", cols))
    if op != "dropout":
        s["w"], s["b"] = 1.0 + 0.1 * normal(cols), 0.1 * normal(cols)
        if op == "join" and case["dir"] == "fwd":
            s["residual"] = features()
        if case["dir"] == "bwd":
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = 1.0 / torch.sqrt((x - s["mean"][:, None]).square().mean(1) + EPS)
            s["y_bar"] = (0.1 * normal(rows, cols)).to(dtype)
            if op == "join":
                s["h_bar"] = (0.1 * normal(rows, cols)).to(dtype)
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import equivariant_gnn_tensor_amd as etpc
    case = s["case"]
    op, fwd = case["op"], case["dir"] == "fwd"
    if op == "norm":
        if fwd:
            return etpc.etpc_layer_norm(s["x"], s["w"], s["b"], eps=EPS)
        return etpc.etpc_layer_norm_backward(s["x"], s["y_bar"], s["mean"], s["rstd"], s["w"])
    if op == "dropout":
        return etpc.etpc_dropout(s["x"], case["p"], s["rng_seed"], s["rng_offset"])
    if op == "irreps_dropout":
        return etpc.etpc_irreps_dropout(case["irreps"], s["x"], case["p"], s["rng_seed"], s["rng_offset"])
    if op == "join":
        if fwd:
            return etpc.etpc_dropout_add_layer_norm(s["x"], s["residual"], s["w"], s["b"], p=case["p"], seed=s["rng_seed"],
                                                    offset=s["rng_offset"], eps=EPS)
        return etpc.etpc_dropout_add_layer_norm_backward(s["x"], s["y_bar"], s["mean"], s["rstd"], s["w"], h_bar=s["h_bar"], p=case["p"],
                                                         seed=s["rng_seed"], offset=s["rng_offset"])
    if fwd:
        return etpc.etpc_irreps_norm(case["irreps"], s["x"], s["w"], s["b"], eps=EPS)
    return etpc.etpc_irreps_norm_backward(case["irreps"], s["x"], s["y_bar"], s["stats"], s["w"])


# ---------------------------------------------------------------- the plain forms

_M32 = 0xFFFFFFFF


def _keep(rows, groups, p, seed, offset):
    """[rows, 8 * groups] truth values: the 16-bit fields of Philox4x32-10 (Salmon, Moraes, Dror and
    Shaw, SC 2011) at counter (group, row, offset), key seed, that are not below 65536 p."""
    c0 = torch.arange(groups, device="cuda")[None, :]
    c1 = torch.arange(rows, device="cuda")[:, None]
    c2 = torch.tensor(offset & _M32, device="cuda")
    c3 = torch.tensor(offset >> 32, device="cuda")
    k0, k1 = seed & _M32, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & _M32) ^ c1 ^ k0, b & _M32, ((a >> 32) & _M32) ^ c3 ^ k1, a & _M32
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    words = torch.stack(torch.broadcast_tensors(c0, c1, c2, c3), -1)
    fields = torch.stack((words & 0xFFFF, words >> 16), -1)
    return fields.reshape(rows, 8 * groups) >= round(p * 65536)


def _scale(p):
    dropped = round(p * 65536)
    return 65536.0 / (65536 - dropped) if dropped < 65536 else 0.0


def _dropped(s, x):
    case = s["case"]
    keep = _keep(x.shape[0], (x.shape[1] + 7) // 8, case["p"], s["rng_seed"], s["rng_offset"])[:, :x.shape[1]]
    return torch.where(keep, x * _scale(case["p"]), torch.zeros((), device="cuda"))


def _norm(x, w, b):
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / torch.sqrt(c.square().mean(1) + EPS)
    return c * rstd[:, None] * w + b, mean, rstd


def _norm_backward(x, y_bar, mean, rstd, w):
    xh = (x - mean[:, None]) * rstd[:, None]
    g = y_bar * w
    x_bar = rstd[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return x_bar, (y_bar * xh).sum(0), y_bar.sum(0)


def _irreps_stats(x, blocks):
    stats = []
    for mul, l, _, at, _ in blocks:
        v = x[:, at:at + mul * (2 * l + 1)]
        mean = v.mean(1) if l == 0 else torch.zeros_like(v[:, 0])
        stats.append(torch.stack((mean, 1.0 / torch.sqrt((v - mean[:, None]).square().mean(1) + EPS)), 1))
    return torch.stack(stats, 1)


def _run_plain(s):
    case = s["case"]
    op, fwd = case["op"], case["dir"] == "fwd"
    x = s["x"].float()
    if op == "norm":
        if fwd:
            y, mean, rstd = _norm(x, s["w"], s["b"])
            return y.to(s["x"].dtype), mean, rstd
        x_bar, w_bar, b_bar = _norm_backward(x, s["y_bar"].float(), s["mean"], s["rstd"], s["w"])
        return x_bar.to(s["x"].dtype), w_bar, b_bar
    if op == "dropout":
        return _dropped(s, x).to(s["x"].dtype)
    if op == "join":
        if fwd:
            h = s["residual"].float() + _dropped(s, x)
            y, mean, rstd = _norm(h, s["w"], s["b"])
            return y.to(s["x"].dtype), h.to(s["x"].dtype), mean, rstd
        h_bar, w_bar, b_bar = _norm_backward(x, s["y_bar"].float(), s["mean"], s["rstd"], s["w"])
        h_bar = h_bar + s["h_bar"].float()
        return _dropped(s, h_bar).to(s["x"].dtype), h_bar.to(s["x"].dtype), w_bar, b_bar
    blocks, dim, channels, biases = s["irreps"]
    rows = x.shape[0]
    if op == "irreps_dropout":
        keep, out, group = _keep(rows, sum((b[0] + 7) // 8 for b in blocks), case["p"], s["rng_seed"], s["rng_offset"]), [], 0
        for mul, l, _, at, _ in blocks:
            v = x[:, at:at + mul * (2 * l + 1)].reshape(rows, 2 * l + 1, mul)
            m = keep[:, None, 8 * group:8 * group + mul]
            out.append(torch.where(m, v * _scale(case["p"]), torch.zeros((), device="cuda")).reshape(rows, -1))
            group += (mul + 7) // 8
        return torch.cat(out, 1)
    if fwd:
        stats, out, bias = _irreps_stats(x, blocks), [], 0
        for k, (mul, l, parity, at, ch) in enumerate(blocks):
            v = x[:, at:at + mul * (2 * l + 1)].reshape(rows, 2 * l + 1, mul)
            y = (v - stats[:, k, 0, None, None]) * stats[:, k, 1, None, None] * s["w"][ch:ch + mul]
            if l == 0 and parity == "e":
                y = y + s["b"][bias:bias + mul]
                bias += mul
            out.append(y.reshape(rows, -1))
        return torch.cat(out, 1), stats
    x_bar, w_bar, b_bar = [], [], []
    for k, (mul, l, parity, at, ch) in enumerate(blocks):
        v = x[:, at:at + mul * (2 * l + 1)].reshape(rows, 2 * l + 1, mul)
        d = s["y_bar"][:, at:at + mul * (2 * l + 1)].reshape(rows, 2 * l + 1, mul)
        rstd = s["stats"][:, k, 1, None, None]
        xh = (v - s["stats"][:, k, 0, None, None]) * rstd
        g = d * s["w"][ch:ch + mul]
        t = g - xh * (g * xh).mean((1, 2), keepdim=True)
        if l == 0:
            t = t - g.mean((1, 2), keepdim=True)
        x_bar.append((rstd * t).reshape(rows, -1))
        w_bar.append((d * xh).sum((0, 1)))
        if l == 0 and parity == "e":
            b_bar.append(d.sum((0, 1)))
    return torch.cat(x_bar, 1), torch.cat(w_bar), torch.cat(b_bar) if b_bar else x.new_zeros(0)


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_fields(rows, groups, seed, offset):
    """Philox4x32-10 on the host: uint16 [rows, groups, 8], the low half of each word first."""
    out = np.empty((rows, groups, 4), np.uint32)
    step = max(1, (1 << 20) // max(1, groups))
    mask, sh = np.uint64(_M32), np.uint64(32)
    for r0 in range(0, rows, step):
        n = min(step, rows - r0)
        shape = (n, groups)
        ctr = [np.broadcast_to(np.arange(groups, dtype=np.uint64), shape),
               np.broadcast_to(np.arange(r0, r0 + n, dtype=np.uint64)[:, None], shape),
               np.full(shape, offset % 2**32, np.uint64), np.full(shape, offset // 2**32, np.uint64)]
        for i in range(10):
            key = [np.uint64((seed % 2**32 + i * 0x9E3779B9) % 2**32), np.uint64((seed // 2**32 + i * 0xBB67AE85) % 2**32)]
            p0, p1 = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
            ctr = [(p1 >> sh) ^ ctr[1] ^ key[0], p1 & mask, (p0 >> sh) ^ ctr[3] ^ key[1], p0 & mask]
        for j in range(4):
            out[r0:r0 + n, :, j] = ctr[j]
    return out.view("<u2")


def _exact_factor(case, s, rows, groups):
    """[rows, 8 * groups] doubles: 0 where dropped, the scale where kept."""
    dropped = int(np.rint(case["p"] * 65536))
    f = _exact_fields(rows, groups, s["rng_seed"], s["rng_offset"]).reshape(rows, 8 * groups)
    return torch.from_numpy((f >= dropped)).cuda().double() * (65536.0 / (65536 - dropped))


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    op, rows, x = case["op"], case["rows"], d["x"]
    if op in ("dropout", "join"):
        factor = _exact_factor(case, s, rows, -(-case["cols"] // 8))[:, :case["cols"]]
    if op == "dropout":
        return x * factor
    if op in ("norm", "join"):
        n = case["cols"]
        if case["dir"] == "fwd":
            h = d["residual"] + x * factor if op == "join" else x
            mean = h.sum(1) / n
            var = (h - mean.unsqueeze(1)).pow(2).sum(1) / n
            rstd = (var + EPS).pow(-0.5)
            y = d["b"] + d["w"] * ((h - mean.unsqueeze(1)) * rstd.unsqueeze(1))
            return (y, h, mean, rstd) if op == "join" else (y, mean, rstd)
        xh = (x - d["mean"].unsqueeze(1)) * d["rstd"].unsqueeze(1)
        g = d["w"] * d["y_bar"]
        a, b = g.sum(1, keepdim=True) / n, (g * xh).sum(1, keepdim=True) / n
        x_bar = d["rstd"].unsqueeze(1) * (g - (a + b * xh))
        w_bar, b_bar = (d["y_bar"] * xh).sum(0), d["y_bar"].sum(0)
        if op == "norm":
            return x_bar, w_bar, b_bar
        x_bar = x_bar + d["h_bar"]
        return x_bar * factor, x_bar, w_bar, b_bar
    blocks, dim, channels, biases = _irreps(case["irreps"])
    if op == "irreps_dropout":
        factor = _exact_factor(case, s, rows, sum(-(-b[0] // 8) for b in blocks))
        y, at = torch.empty_like(x), 0
        for mul, l, _, off, _ in blocks:
            for m in range(2 * l + 1):
                y[:, off + m * mul:off + (m + 1) * mul] = x[:, off + m * mul:off + (m + 1) * mul] * factor[:, at:at + mul]
            at += -(-mul // 8) * 8
        return y
    out, stats = torch.zeros_like(x), torch.zeros(rows, len(blocks), 2, dtype=torch.float64, device="cuda")
    w_bar, b_bar, bias = x.new_zeros(channels), x.new_zeros(biases), 0
    for k, (mul, l, parity, off, ch) in enumerate(blocks):
        width = mul * (2 * l + 1)
        part, gain = slice(off, off + width), d["w"][ch:ch + mul].repeat(2 * l + 1)
        v = x[:, part]
        if case["dir"] == "fwd":
            mean = v.sum(1, keepdim=True) / mul if l == 0 else torch.zeros(rows, 1, dtype=torch.float64, device="cuda")
            rstd = ((v - mean).pow(2).sum(1, keepdim=True) / width + EPS).pow(-0.5)
            out[:, part] = gain * ((v - mean) * rstd)
            stats[:, k, 0:1], stats[:, k, 1:2] = mean, rstd
        else:
            mean, rstd = d["stats"][:, k, 0:1], d["stats"][:, k, 1:2]
            xh, yb = (v - mean) * rstd, d["y_bar"][:, part]
            a = (yb * gain).sum(1, keepdim=True) / width if l == 0 else 0.0
            out[:, part] = rstd * (yb * gain - a - xh * ((yb * gain * xh).sum(1, keepdim=True) / width))
            w_bar[ch:ch + mul] = (yb * xh).sum(0).reshape(2 * l + 1, mul).sum(0)
        if l == 0 and parity == "e":
            if case["dir"] == "fwd":
                out[:, part] += d["b"][bias:bias + mul]
            else:
                b_bar[bias:bias + mul] = d["y_bar"][:, part].sum(0)
            bias += mul
    return (out, stats) if case["dir"] == "fwd" else (out, w_bar, b_bar)


def work(case):
    op, rows, fwd = case["op"], case["rows"], case["dir"] == "fwd"
    if op.startswith("irreps"):
        blocks, dim, channels, biases = _irreps(case["irreps"])
        n = rows * dim
        if op == "irreps_dropout":
            return {"bytes": 8 * n, "flops": n}
        side = 8 * rows * len(blocks)
        if fwd:
            return {"bytes": 8 * n + side + 4 * (channels + biases), "flops": 6 * n}
        return {"bytes": 12 * n + side + 4 * (2 * channels + biases), "flops": 12 * n}
    size, n, cols = (4 if case["dtype"] == "f32" else 2), rows * case["cols"], case["cols"]
    if op == "dropout":
        return {"bytes": 2 * size * n, "flops": n}
    if fwd:
        return {"bytes": (2 if op == "norm" else 4) * size * n + 8 * rows + 8 * cols, "flops": (7 if op == "norm" else 9) * n}
    return {"bytes": (3 if op == "norm" else 5) * size * n + 8 * rows + 12 * cols, "flops": (12 if op == "norm" else 14) * n}
