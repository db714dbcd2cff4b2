"""Timed cases of the feed-forward operators: a dense layer with bias, activation and residual,
the gated residual join between two norms, and the global gradient norm with clipping.

Each case runs one operator in one direction.  `own = False` computes it with elementary
torch operations in 32 bits; `own = True` calls this package.  `exact` gives the same
outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5
ACTS = ("none", "relu", "silu", "gelu", "tanh")


def listed():
    return [
        # one row of invariants through a readout's hidden layer at inference: latency
        dict(name="linear_one_row", op="linear", dir="fwd", dtype="f32", rows=1, n_in=1024, n_out=1024, act="silu", layout="io",
             residual=False, pitch=0),
        # the radial network's hidden layer on the 214980 edges of the 4096-atom graph
        dict(name="linear_edges_fwd", op="linear", dir="fwd", dtype="bf16", rows=214980, n_in=64, n_out=64, act="silu", layout="io",
             residual=False, pitch=0),
        # its gradient
        dict(name="linear_edges_bwd", op="linear", dir="bwd", dtype="bf16", rows=214980, n_in=64, n_out=64, act="silu", layout="io",
             pitch=0),
        # the widening layer of a feed-forward block on the invariants of 511 cells of 128 atoms: throughput
        dict(name="linear_wide_fwd", op="linear", dir="fwd", dtype="bf16", rows=65408, n_in=1024, n_out=4096, act="gelu", layout="oi",
             residual=False, pitch=0),
        # the gradient of the narrowing layer of that block
        dict(name="linear_wide_bwd", op="linear", dir="bwd", dtype="f16", rows=65408, n_in=4096, n_out=1024, act="none", layout="oi",
             pitch=0),
        # odd sizes with a residual, out of rows that hold other columns too
        dict(name="linear_odd_fwd", op="linear", dir="fwd", dtype="f32", rows=4097, n_in=2047, n_out=511, act="silu", layout="io",
             residual=True, pitch=5),
        # invariants of a small graph at inference: latency
        dict(name="join_small", op="join", dir="fwd", dtype="f32", rows=64, cols=64, gate=True, pitch=0),
        # invariants of 511 cells between two blocks, in training
        dict(name="join_large_fwd", op="join", dir="fwd", dtype="bf16", rows=65408, cols=1024, gate=True, pitch=0),
        # the gradient at odd sizes
        dict(name="join_odd_bwd", op="join", dir="bwd", dtype="f32", rows=4097, cols=2047, gate=True, pitch=0),
        # the parameters of one block: latency
        dict(name="clip_small", op="clip", dtype="f32", tensors=12, total=20000, spread=0.8, clip=0.5, align=16),
        # a network's parameters of all sizes, weights in 16 bits, gains and biases in 32
        dict(name="clip_model", op="clip", dtype="mixed", tensors=260, total=1 << 26, spread=2.0, clip=0.5, align=16),
        # the norm alone, over large 16-bit gradients
        dict(name="norm_large", op="norm", dtype="bf16", tensors=24, total=3 << 27, spread=1.0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["linear"] * 4 + ["join"] * 2 + ["clip", "norm"])
    if op in ("clip", "norm"):
        tensors = _log(rng, 1, 400)
        case = dict(op=op, dtype=rng.choice(["f32", "bf16", "f16", "mixed"]), tensors=tensors,
                    total=_log(rng, max(16, tensors), 1 << (26 if op == "clip" else 28)), spread=round(rng.uniform(0.0, 2.5), 3))
        if op == "clip":
            case["clip"], case["align"] = rng.choice([0.1, 0.5, 2.0]), rng.choice([16, 16, 1])
        return case
    dtype, direction = rng.choice(["f32", "bf16", "f16"]), rng.choice(["fwd", "bwd"])
    if op == "join":
        cols = _log(rng, 4, 16384)
        if rng.random() < 0.5 and cols > 16:
            cols = cols // 16 * 16
        rows = _log(rng, 1, min(1 << 18, (1 << (25 if direction == "fwd" else 24)) // cols))
        return dict(op=op, dir=direction, dtype=dtype, rows=rows, cols=cols, gate=rng.random() < 0.8, pitch=rng.choice([0, 0, 8, 5]))
    n_in, n_out = _log(rng, 1, 4096), _log(rng, 1, 4096)
    if rng.random() < 0.6:   # multiples of eight are usual, others occur
        n_in, n_out = max(8, n_in // 8 * 8), max(8, n_out // 8 * 8)
    most = min((1 << (34 if dtype == "f32" else 37)) // (n_in * n_out), (1 << 27) // (n_in + n_out), 1 << 18)
    case = dict(op=op, dir=direction, dtype=dtype, rows=_log(rng, 1, most), n_in=n_in, n_out=n_out, act=rng.choice(ACTS),
                layout=rng.choice(["io", "oi"]), pitch=rng.choice([0, 0, 0, 8, 5]))
    if direction == "fwd":
        case["residual"] = rng.random() < 0.4
    return case


def _sizes(case):
    """Sizes of the gradient tensors: `tensors` of them with `total` elements, log-normally spread."""
    n, total, rng = case["tensors"], case["total"], random.Random(case["tensors"] * 1000003 + case["total"])
    share = [math.exp(rng.gauss(0.0, case["spread"])) for _ in range(n)]
    scale = (total - n) / sum(share)
    sizes = [1 + int(v * scale) for v in share]
    sizes[-1] += total - sum(sizes)
    return sizes


def _tensor_dtype(case, k):
    return DTYPES[case["dtype"] if case["dtype"] != "mixed" else ("bf16" if k % 2 == 0 else "f32")]


def _buckets(case, grads):
    """One flat buffer for each type, and every tensor's place in them (from a multiple of `align` on)."""
    at, places = {}, []
    for g in grads:
        places.append(at.get(g.dtype, 0))
        at[g.dtype] = places[-1] + -(-g.numel() // case["align"]) * case["align"]
    flats = {t: torch.zeros(n, dtype=t, device="cuda") for t, n in at.items()}
    return list(flats.values()), [flats[g.dtype][p:p + g.numel()] for g, p in zip(grads, places)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s, op = dict(case=case), case["op"]
    if op in ("clip", "norm"):
        level = 0.5 + torch.rand(case["tensors"], generator=gen, device="cuda")   # tensors have levels of their own
        s["grads"] = [(0.1 * level[k] * normal(n)).to(_tensor_dtype(case, k)) for k, n in enumerate(_sizes(case))]
        if op == "clip":
            s["max_norm"] = case["clip"] * 0.1 * math.sqrt(case["total"])
            s["flats"], s["outs"] = _buckets(case, s["grads"])
        return s
    rows, dtype = case["rows"], DTYPES[case["dtype"]]

    def matrix(values, pitch=0):
        """The values in the case's type, as the first columns of wider rows."""
        if pitch == 0:
            return values.to(dtype)
        full = torch.empty(values.shape[0], values.shape[1] + pitch, device="cuda", dtype=dtype).fill_(0.25)
        full[:, :values.shape[1]] = values.to(dtype)
        return full[:, :values.shape[1]]

    if op == "linear":
        n_in, n_out = case["n_in"], case["n_out"]
        s["x"] = matrix(normal(rows, n_in) + 0.2 * normal(n_in), case["pitch"])
        w = matrix(normal(n_in, n_out) / math.sqrt(n_in))
        s["w"] = w if case["layout"] == "io" else w.t().contiguous().t()   # either axis contiguous
        s["b"] = 0.1 * normal(n_out)
        if case["dir"] == "fwd":
            s["residual"] = matrix(normal(rows, n_out)) if case["residual"] else None
        else:
            s["y_bar"] = matrix(0.1 * normal(rows, n_out) + 0.02 * normal(n_out))
            s["z"] = matrix(s["x"].float() @ s["w"].float() + s["b"]) if case["act"] != "none" else None
        return s
    cols = case["cols"]
    level = 0.5 + torch.rand(rows, 1, generator=gen, device="cuda")
    s["x"] = matrix((normal(rows, cols) + 0.3 * normal(cols)) * level, case["pitch"])
    s["residual"] = matrix(normal(rows, cols) + 0.3 * normal(cols))
    s["gate"] = matrix(normal(rows, cols)) if case["gate"] else None
    for name in ("w1", "w2"):
        s[name] = 1.0 + 0.1 * normal(cols)
    for name in ("b1", "b2"):
        s[name] = 0.1 * normal(cols)
    s["scale"] = 0.5 + 0.1 * normal(cols)
    if case["dir"] == "bwd":
        _, h, s["stats"] = _join(s)
        s["h"] = h.to(dtype)
        s["y_bar"], s["h_bar"] = matrix(0.1 * normal(rows, cols)), matrix(0.1 * normal(rows, cols))
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import equivariant_gnn_tensor_amd as etpc
    case = s["case"]
    op = case["op"]
    if op == "norm":
        return etpc.etpc_grad_norm(s["grads"])
    if op == "clip":
        return etpc.etpc_clip_grad_norm(s["grads"], s["max_norm"], outs=s["outs"]), s["flats"]
    if op == "linear":
        if case["dir"] == "fwd":
            y, z = etpc.etpc_linear(s["x"], s["w"], s["b"], residual=s["residual"], act=case["act"])
            return y if z is None else (y, z)
        return etpc.etpc_linear_backward(s["x"], s["w"], s["y_bar"], z=s["z"], act=case["act"])
    if case["dir"] == "fwd":
        return etpc.etpc_norm_gate_add_norm(s["x"], gate=s["gate"], residual=s["residual"], w1=s["w1"], b1=s["b1"], scale=s["scale"],
                                            w2=s["w2"], b2=s["b2"], eps=EPS)
    return tuple(t for t in etpc.etpc_norm_gate_add_norm_backward(
        s["x"], s["h"], s["y_bar"], s["stats"], gate=s["gate"], w1=s["w1"], b1=s["b1"], scale=s["scale"], w2=s["w2"],
        h_bar=s["h_bar"]) if t is not None)


# ---------------------------------------------------------------- the plain forms


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros((), device="cuda"))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    return torch.tanh(z) if act == "tanh" else z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return 1.0 - torch.tanh(z).square()


def _normed(x):
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / torch.sqrt(c.square().mean(1) + EPS)
    return c * rstd[:, None], mean, rstd


def _normed_backward(xh, g, rstd):
    return rstd[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))


def _join(s):
    xh, mean, rstd = _normed(s["x"].float())
    n = xh * s["w1"] + s["b1"]
    if s["gate"] is not None:
        n = n / (1.0 + torch.exp(-s["gate"].float()))
    h = s["residual"].float() + s["scale"] * n
    hh, mean_h, rstd_h = _normed(h)
    return hh * s["w2"] + s["b2"], h, torch.stack((mean, rstd, mean_h, rstd_h), 1)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op in ("clip", "norm"):
        norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
        if op == "norm":
            return norm
        factor = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
        for g, out in zip(s["grads"], s["outs"]):
            out.copy_(g.float() * factor)
        return norm, s["flats"]
    dtype = s["x"].dtype
    if op == "linear":
        x, w = s["x"].float(), s["w"].float()
        if case["dir"] == "fwd":
            z = x @ w + s["b"]
            y = _act(z, case["act"])
            if s["residual"] is not None:
                y = y + s["residual"].float()
            return y.to(dtype) if case["act"] == "none" else (y.to(dtype), z.to(dtype))
        z_bar = s["y_bar"].float()
        if case["act"] != "none":
            z_bar = z_bar * _act_slope(s["z"].float(), case["act"])
        return (z_bar @ w.t()).to(dtype), (x.t() @ z_bar).to(dtype), z_bar.sum(0)
    if case["dir"] == "fwd":
        y, h, stats = _join(s)
        return y.to(dtype), h.to(dtype), stats
    st = s["stats"]
    xh = (s["x"].float() - st[:, 0:1]) * st[:, 1:2]
    hh = (s["h"].float() - st[:, 2:3]) * st[:, 3:4]
    y_bar = s["y_bar"].float()
    d = s["h_bar"].float() + _normed_backward(hh, y_bar * s["w2"], st[:, 3])
    n = xh * s["w1"] + s["b1"]
    p = 1.0 / (1.0 + torch.exp(-s["gate"].float())) if s["gate"] is not None else torch.ones((), device="cuda")
    u = d * s["scale"] * p
    x_bar = _normed_backward(xh, u * s["w1"], st[:, 1])
    gates = ((u * n * (1.0 - p)).to(dtype),) if s["gate"] is not None else ()
    return (x_bar.to(dtype), *gates, d.to(dtype), (u * xh).sum(0), u.sum(0), (d * p * n).sum(0), (y_bar * hh).sum(0), y_bar.sum(0))


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_act(z, act):
    """Activation and slope."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), torch.heaviside(z, torch.zeros_like(z))
    if act == "silu":
        p = torch.special.expit(z)
        return z * p, p + z * p * torch.special.expit(-z)
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(z * z / -2) / (2 * math.pi) ** 0.5
    return torch.tanh(z), torch.cosh(z).pow(-2)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("clip", "norm"):
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g, dtype=torch.float64)) ** 2 for g in s["grads"]))
        value = torch.tensor(norm, dtype=torch.float64, device="cuda")
        if op == "norm":
            return value
        factor = min(1.0, s["max_norm"] / (norm + 1e-6))
        wide, parts = [torch.zeros_like(f, dtype=torch.float64) for f in s["flats"]], {f.dtype: k for k, f in enumerate(s["flats"])}
        for g, out in zip(s["grads"], s["outs"]):
            wide[parts[g.dtype]][out.storage_offset():out.storage_offset() + g.numel()] = factor * g.double()
        return value, wide
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    x, n = d["x"], d["x"].shape[1]
    if op == "linear":
        if case["dir"] == "fwd":
            z = torch.addmm(d["b"].unsqueeze(0), x, d["w"])
            y = _exact_act(z, case["act"])[0]
            y = y + d["residual"] if "residual" in d else y
            return y if case["act"] == "none" else (y, z)
        z_bar = d["y_bar"] * _exact_act(d["z"], case["act"])[1] if "z" in d else d["y_bar"]
        return torch.mm(z_bar, d["w"].t()), torch.mm(x.t(), z_bar), z_bar.sum(0)
    p = torch.special.expit(d["gate"]) if "gate" in d else torch.ones_like(x)
    if case["dir"] == "fwd":
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        rstd = (var + EPS).rsqrt()
        h = d["residual"] + d["scale"] * p * (d["b1"] + d["w1"] * (x - mean) * rstd)
        var_h, mean_h = torch.var_mean(h, 1, correction=0, keepdim=True)
        rstd_h = (var_h + EPS).rsqrt()
        return d["b2"] + d["w2"] * (h - mean_h) * rstd_h, h, torch.cat((mean, rstd, mean_h, rstd_h), 1)
    mean, rstd, mean_h, rstd_h = d["stats"].unsqueeze(2).unbind(1)
    hh, xh = (d["h"] - mean_h) * rstd_h, (x - mean) * rstd
    g = d["w2"] * d["y_bar"]
    res = d["h_bar"] + rstd_h * (g - (g.sum(1, keepdim=True) + hh * (g * hh).sum(1, keepdim=True)) / n)
    branch = d["b1"] + d["w1"] * xh
    u = res * (d["scale"] * p)
    g = d["w1"] * u
    x_bar = rstd * (g - (g.sum(1, keepdim=True) + xh * (g * xh).sum(1, keepdim=True)) / n)
    out = [x_bar] + ([res * d["scale"] * branch * p * torch.special.expit(-d["gate"])] if "gate" in d else [])
    return (*out, res, (u * xh).sum(0), u.sum(0), (res * p * branch).sum(0), (d["y_bar"] * hh).sum(0), d["y_bar"].sum(0))


def work(case):
    op = case["op"]
    if op in ("clip", "norm"):
        size = sum(n * _tensor_dtype(case, k).itemsize for k, n in enumerate(_sizes(case)))
        return {"bytes": (2 if op == "clip" else 1) * size, "flops": (3 if op == "clip" else 2) * case["total"]}
    size, rows = (4 if case["dtype"] == "f32" else 2), case["rows"]
    if op == "linear":
        a, b = case["n_in"], case["n_out"]
        kept = 1 if case["act"] != "none" else 0
        if case["dir"] == "fwd":
            return {"bytes": size * (rows * a + a * b + rows * b * (1 + kept + (1 if case["residual"] else 0))) + 4 * b,
                    "flops": 2 * rows * a * b}
        return {"bytes": 2 * size * (rows * a + a * b) + size * rows * b * (1 + kept) + 4 * b, "flops": 4 * rows * a * b}
    n, gate = rows * case["cols"], 1 if case["gate"] else 0
    if case["dir"] == "fwd":
        return {"bytes": size * n * (4 + gate) + 16 * rows + 20 * case["cols"], "flops": 20 * n}
    return {"bytes": size * n * (6 + 2 * gate) + 16 * rows + 36 * case["cols"], "flops": 36 * n}
