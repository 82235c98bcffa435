"""The gated feed-forward block's operators on their working range: inputs, plain forms, the library's calls and exact
values.

The operators are a gated linear layer (both projections, the activation and the product), its gradients, the layer norm
with the residual's addition (its output in the input's type or in 8 bits with a scale a row), its gradients, and the
clipping of a model's gradients by their common norm.  ``run`` computes an operator in elementary torch operations in 32
bits, or, with ``own`` set, through the calls that a user makes of the library.
"""
import math

import torch

own = False

EPS = 1e-5            # the norm's epsilon
CLIP_EPS = 1e-6       # added to the gradients' norm before it divides
E4M3_MAX = 448.0      # largest finite value of the 8-bit type
AMAX_FLOOR = 1e-30    # a row of zeros gets the scale AMAX_FLOOR / E4M3_MAX

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
ACTIVATIONS = ("silu", "silu", "gelu", "gelu_erf", "relu", "none")


def _gated(name, dtype, m, n, k, act="silu", bias=False, preact=False, w_kn=False):
    return {"name": name, "op": "gated", "dtype": dtype, "m": m, "n": n, "k": k, "act": act, "bias": bias,
            "preact": preact, "w_kn": w_kn}


def _clip(name, dtype, layers, width, hidden, max_norm=1.0):
    return {"name": name, "op": "clip", "dtype": dtype, "layers": layers, "width": width, "hidden": hidden,
            "max_norm": max_norm}


def listed():
    return [
        # one token of a decoding step: both weights are read once, latency counts
        _gated("gated_token_bf16", "bf16", 1, 11264, 4096),
        # a decoding batch on 8-bit weights and activations
        _gated("gated_batch_e4m3", "e4m3", 64, 8192, 4096),
        # a training step's two projections, which keep both pre-activations for the gradients
        _gated("gated_train_bf16", "bf16", 4096, 11264, 4096, preact=True),
        # a full-precision block of ragged sizes: neither rows nor columns a multiple of any tile or vector
        _gated("gated_ragged_f32", "f32", 1000, 1369, 1001, act="gelu", bias=True),
        # gradients of a training step's block
        {"name": "gated_backward_bf16", "op": "gated_backward", "dtype": "bf16", "m": 4096, "n": 8192, "k": 4096,
         "act": "silu", "bias": False, "w_kn": False},
        # gradients of a small full-precision block of odd sizes
        {"name": "gated_backward_ragged_f32", "op": "gated_backward", "dtype": "f32", "m": 500, "n": 777, "k": 1001,
         "act": "gelu", "bias": True, "w_kn": False},
        # the norm before a projection in a decoding step, written as the 8-bit row that the product reads
        {"name": "layernorm_token_e4m3", "op": "layernorm", "dtype": "bf16", "rows": 1, "d": 4096, "bias": True,
         "residual": True, "quantize": True},
        # the norm of a prefill or a training step
        {"name": "layernorm_prefill_bf16", "op": "layernorm", "dtype": "bf16", "rows": 8192, "d": 8192, "bias": True,
         "residual": True, "quantize": False},
        # its gradients in a training step, joined with the residual stream's
        {"name": "layernorm_backward_bf16", "op": "layernorm_backward", "dtype": "bf16", "rows": 8192, "d": 4096,
         "bias": True, "stream_grad": True},
        # the same of an odd width in full precision, with few rows to sum the weight's gradient over
        {"name": "layernorm_backward_odd_f32", "op": "layernorm_backward", "dtype": "f32", "rows": 1000, "d": 1001,
         "bias": True, "stream_grad": False},
        # all gradients of a model of 24 gated blocks, 168 tensors of 302 million elements
        _clip("clip_model_bf16", "bf16", 24, 1024, 4096),
        # a small model's, where the launches count
        _clip("clip_small_f32", "f32", 4, 256, 1000),
    ]


def _size(rng, low, high):
    """Log-uniform; often a multiple of 64 where it is large enough, as widths are, else any number."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if v >= 128 and rng.random() < 0.6:
        v = v // 64 * 64
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_backward", "layernorm", "layernorm_backward", "clip"])
    if op == "gated":
        c = _gated("", rng.choice(["f32", "bf16", "bf16", "f16", "e4m3"]), _size(rng, 1, 4096), _size(rng, 16, 8192),
                   _size(rng, 16, 4096), act=rng.choice(ACTIVATIONS), bias=rng.random() < 0.4,
                   preact=rng.random() < 0.4)
        c["w_kn"] = c["dtype"] != "e4m3" and rng.random() < 0.25
    elif op == "gated_backward":
        c = {"op": op, "dtype": rng.choice(["f32", "bf16", "bf16", "f16"]), "m": _size(rng, 1, 4096),
             "n": _size(rng, 16, 8192), "k": _size(rng, 16, 4096), "act": rng.choice(ACTIVATIONS),
             "bias": rng.random() < 0.5, "w_kn": rng.random() < 0.25}
    elif op == "clip":
        c = _clip("", rng.choice(["f32", "bf16", "f16", "mixed"]), 1, _size(rng, 16, 1024), _size(rng, 16, 4096),
                  max_norm=rng.choice([0.1, 1.0, 1.0, 1e4]))
        # as many layers as the largest listed list has bytes for
        c["layers"] = min(_size(rng, 1, 24), 24 * 2 * 1024 * 4096 // (4 * c["width"] * c["hidden"]) or 1)
    else:
        d = _size(rng, 16, 8192)
        c = {"op": op, "dtype": rng.choice(["f32", "bf16", "bf16", "f16"]), "rows": _size(rng, 1, 16384), "d": d,
             "bias": rng.random() < 0.8}
        if c["dtype"] == "f32" or d > 4096:
            c["rows"] = min(c["rows"], 4096)
        if op == "layernorm":
            c |= {"residual": rng.random() < 0.7, "quantize": rng.random() < 0.4}
        else:
            c |= {"stream_grad": rng.random() < 0.7}
    c.pop("name", None)
    return c


# ---------------------------------------------------------------------------------------------------- inputs


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def _activations(g, rows, d):
    """Rows of different size about a common offset, with a few columns far larger than the others, as hidden states
    have."""
    x = _normal(g, rows, d) + _normal(g, d, std=0.3) + 0.1
    x *= torch.exp(_normal(g, rows, 1, std=0.3))
    big = torch.randint(0, d, (max(1, d // 512),), generator=g, device="cuda")
    x[:, big] *= 12.0
    return x


def _to_e4m3(x):
    a = x.abs().amax(1).clamp_min(AMAX_FLOOR)
    q = (x * (E4M3_MAX / a)[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q, a / E4M3_MAX


def _shapes(case):
    """The parameters of every layer: a norm's weight and bias, gate, up and down projections, the first two's biases."""
    w, h = case["width"], case["hidden"]
    return [(w,), (w,), (h, w), (h, w), (w, h), (h,), (h,)] * case["layers"]


def _type(case, shape):
    if case["dtype"] == "mixed":     # norms and biases kept in 32 bits beside 16-bit matrices
        return "bf16" if len(shape) == 2 else "f32"
    return case["dtype"]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    if case["op"] in ("gated", "gated_backward"):
        m, n, k = case["m"], case["n"], case["k"]
        s["out"] = out = DTYPES["bf16" if case["dtype"] == "e4m3" else case["dtype"]]
        s["x"], s["x_scale"] = _activations(g, m, k), None
        if case["dtype"] == "e4m3":
            s["x"], s["x_scale"] = _to_e4m3(s["x"])
        else:
            s["x"] = s["x"].to(out)
        for name in ("gate", "up"):
            w = _normal(g, n, k, std=k ** -0.5)
            s["s_" + name] = None
            if case["dtype"] == "e4m3":
                s["w_" + name], s["s_" + name] = _to_e4m3(w)
            else:
                # a weight stored with the outputs contiguous is the transposed view of a K x N matrix
                s["w_" + name] = w.to(out).t().contiguous().t() if case["w_kn"] else w.to(out)
            s["b_" + name] = _normal(g, n, std=0.2).to(out) if case["bias"] else None
            if case["op"] == "gated_backward":
                s["z_" + name] = _normal(g, m, n).to(out)
        if case["op"] == "gated_backward":
            s["dh"] = _normal(g, m, n).to(out)
        return s
    if case["op"] == "clip":
        # parameters' gradients differ in size, matrices' are the larger part of the norm
        shapes = _shapes(case)
        for key in ("grads", "out"):
            # views of one buffer a type, one behind the other, as training loops keep them
            s["flat_" + key] = {}
            views = {}
            for t in sorted({_type(case, shape) for shape in shapes}):
                sizes = [math.prod(shape) for shape in shapes if _type(case, shape) == t]
                s["flat_" + key][t] = torch.empty(sum(sizes), dtype=DTYPES[t], device="cuda")
                views[t] = list(s["flat_" + key][t].split(sizes))
            s[key] = [views[_type(case, shape)].pop(0).view(shape) for shape in shapes]
        for i, t in enumerate(s["grads"]):
            t.copy_(_normal(g, *t.shape, std=2e-3) * (1 + i % 7))
        return s
    rows, d, t = case["rows"], case["d"], DTYPES[case["dtype"]]
    s["x"] = _activations(g, rows, d).to(t)
    s["w"] = (1.0 + _normal(g, d, std=0.1)).to(t)
    if case["op"] == "layernorm":
        s["b"] = _normal(g, d, std=0.1).to(t) if case["bias"] else None
        s["r"] = _activations(g, rows, d).to(t) if case["residual"] else None
    else:
        s["dy"] = _normal(g, rows, d).to(t)
        s["ds"] = _normal(g, rows, d).to(t) if case["stream_grad"] else None
        x = s["x"].double()
        s["mean"] = x.mean(1)
        s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + EPS).float()
        s["mean"] = s["mean"].float()
    return s


# ---------------------------------------------------------------------------------------------------- plain forms


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "gelu_erf":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if act == "gelu_erf":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _project(s, name):
    x, w = s["x"].float(), s["w_" + name].float()
    if s["x_scale"] is not None:
        x, w = x * s["x_scale"][:, None], w * s["s_" + name][:, None]
    z = x @ w.t()
    return z if s["b_" + name] is None else z + s["b_" + name].float()


def _plain(s):
    if s["op"] == "gated":
        zg, zu = _project(s, "gate"), _project(s, "up")
        h = (_act(zg, s["act"]) * zu).to(s["out"])
        return (h, zg.to(s["out"]), zu.to(s["out"])) if s["preact"] else h
    if s["op"] == "gated_backward":
        dh, zg, zu, x = s["dh"].float(), s["z_gate"].float(), s["z_up"].float(), s["x"].float()
        dg, du = dh * zu * _act_grad(zg, s["act"]), dh * _act(zg, s["act"])
        dx = dg @ s["w_gate"].float() + du @ s["w_up"].float()
        out = [dx, dg.t() @ x, du.t() @ x] + ([dg.sum(0), du.sum(0)] if s["bias"] else [])
        return [t.to(s["out"]) for t in out]
    if s["op"] == "clip":
        # (long sums: in 64 bits)
        parts = [t.float().square().sum(dtype=torch.float64) for t in s["grads"]]
        norm = torch.stack(parts).sum().sqrt()
        coef = (s["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0).float()
        scaled = [(t.float() * coef).to(t.dtype) for t in s["grads"]]
        return norm.float(), {t: torch.cat([x.flatten() for x in scaled if x.dtype == flat.dtype])
                              for t, flat in s["flat_grads"].items()}
    if s["op"] == "layernorm":
        h = s["x"].float()
        if s["r"] is not None:
            h = h + s["r"].float()
        mean = h.mean(1)
        c = h - mean[:, None]
        rstd = torch.rsqrt(c.square().mean(1) + EPS)
        y = c * rstd[:, None] * s["w"].float()
        if s["b"] is not None:
            y = y + s["b"].float()
        h = h.to(s["x"].dtype)
        return (*_to_e4m3(y), h, mean, rstd) if s["quantize"] else (y.to(s["x"].dtype), h, mean, rstd)
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    n = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["w"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    if s["ds"] is not None:
        dx = dx + s["ds"].float()
    out = [dx, (dy * n).sum(0)] + ([dy.sum(0)] if s["bias"] else [])
    return [t.to(s["x"].dtype) for t in out]


def run(state):
    s = state
    if not own:
        return _plain(s)
    import dense_fp32_matrix_sgemm_gb300 as sg
    if s["op"] == "gated":
        return sg.gated_linear(s["x"], s["w_gate"], s["w_up"], s["b_gate"], s["b_up"], activation=s["act"],
                               x_scale=s["x_scale"], gate_scale=s["s_gate"], up_scale=s["s_up"],
                               save_preact=s["preact"])
    if s["op"] == "gated_backward":
        out = sg.gated_linear_backward(s["dh"], s["x"], s["w_gate"], s["w_up"], s["z_gate"], s["z_up"],
                                       activation=s["act"], need_db=s["bias"])
        return list(out if s["bias"] else out[:3])
    if s["op"] == "clip":
        return sg.clip_grad_norm(s["grads"], s["max_norm"], eps=CLIP_EPS, out=s["out"]), s["flat_out"]
    if s["op"] == "layernorm":
        return sg.add_layernorm(s["x"], s["w"], s["b"], s["r"], eps=EPS, quantize=s["quantize"])
    out = sg.add_layernorm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"], s["ds"], need_dbias=s["bias"])
    return list(out if s["bias"] else out[:2])


# ---------------------------------------------------------------------------------------------------- cost and exact values


def work(case):
    if case["op"] == "clip":
        sizes = [(math.prod(shape), BYTES[_type(case, shape)]) for shape in _shapes(case)]
        return {"bytes": sum(2 * n * e for n, e in sizes) + 4, "flops": sum(3 * n for n, _ in sizes)}
    e = BYTES[case["dtype"]]
    if case["op"] == "gated":
        m, n, k = case["m"], case["n"], case["k"]
        o = 2 if case["dtype"] == "e4m3" else e
        scales = 4 * (m + 2 * n) if case["dtype"] == "e4m3" else 0
        moved = e * (m * k + 2 * n * k) + scales + o * m * n * (1 + 2 * case["preact"]) + 2 * o * n * case["bias"]
        return {"bytes": moved, "flops": 4 * m * n * k}
    if case["op"] == "gated_backward":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": e * (2 * m * k + 4 * n * k + 3 * m * n + 2 * n * case["bias"]), "flops": 8 * m * n * k}
    r, d = case["rows"], case["d"]
    if case["op"] == "layernorm":
        stream = 2 * e if case["residual"] else 0      # the residual read and the sum written
        y = r * d + 4 * r if case["quantize"] else r * d * e
        return {"bytes": r * d * (e + stream) + y + e * d * (1 + case["bias"]) + 8 * r,
                "flops": (8 + 3 * case["quantize"]) * r * d}
    return {"bytes": r * d * e * (3 + case["stream_grad"]) + e * d * (2 + case["bias"]) + 8 * r, "flops": 14 * r * d}


def exact(case, seed):
    """The same outputs in 64 bits, not rounded to the output's type (8-bit codes: the quotients they round)."""
    s = prepare(case, seed)
    if case["op"] == "clip":
        wide = {t: flat.to(torch.float64) for t, flat in s["flat_grads"].items()}
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(flat) for flat in wide.values()]))
        scale = min(1.0, case["max_norm"] / (float(norm) + CLIP_EPS))
        return norm, {t: flat.mul_(scale) for t, flat in wide.items()}
    v = {k: t.to(torch.float64) for k, t in s.items() if isinstance(t, torch.Tensor)}
    if case["op"] == "layernorm":
        h = v["x"] + v["r"] if case["residual"] else v["x"]
        var, mean = torch.var_mean(h, dim=1, correction=0)
        inv = (var + EPS) ** -0.5
        y = torch.einsum("rd,r,d->rd", h - mean.unsqueeze(1), inv, v["w"])
        y = y + v["b"] if case["bias"] else y
        if not case["quantize"]:
            return y, h, mean, inv
        top = y.abs().max(dim=1).values.clamp(min=AMAX_FLOOR)
        return y / top.unsqueeze(1) * E4M3_MAX, top / E4M3_MAX, h, mean, inv
    if case["op"] == "layernorm_backward":
        d = case["d"]
        n = (v["x"] - v["mean"].unsqueeze(1)) * v["rstd"].unsqueeze(1)     # the normalised rows
        g = v["dy"] * v["w"]
        dx = v["rstd"].unsqueeze(1) * (g - (g.sum(dim=1, keepdim=True) + n * torch.einsum("rd,rd->r", g, n).unsqueeze(1)) / d)
        if case["stream_grad"]:
            dx = v["ds"] + dx
        grads = [dx, torch.einsum("rd,rd->d", v["dy"], n)]
        return grads + [torch.ones(len(n), dtype=n.dtype, device=n.device) @ v["dy"]] if case["bias"] else grads

    def slope_and_value(z):
        if case["act"] == "relu":
            return (z > 0).double(), z.clamp(min=0)
        if case["act"] == "silu":
            p = torch.sigmoid(z)
            return p + z * p * (1 - p), z * p
        if case["act"] == "gelu_erf":
            p = torch.special.ndtr(z)
            return p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi), z * p
        if case["act"] == "gelu":
            u = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
            p = torch.sigmoid(u)                         # (1 + tanh(u / 2)) / 2
            return p + z * p * (1 - p) * math.sqrt(8 / math.pi) * (1 + 0.134145 * z * z), z * p
        return torch.ones_like(z), z

    if case["op"] == "gated":
        z = {}
        for name in ("gate", "up"):
            z[name] = torch.matmul(v["x"], v["w_" + name].transpose(0, 1))
            if case["dtype"] == "e4m3":
                z[name] = z[name] * v["x_scale"].unsqueeze(1) * v["s_" + name]
            if case["bias"]:
                z[name] = z[name] + v["b_" + name]
        h = slope_and_value(z["gate"])[1] * z["up"]
        return (h, z["gate"], z["up"]) if case["preact"] else h
    slope, value = slope_and_value(v["z_gate"])
    both = torch.cat([v["dh"] * v["z_up"] * slope, v["dh"] * value], dim=1)      # gradients of both pre-activations
    dx = torch.matmul(both, torch.cat([v["w_gate"], v["w_up"]], dim=0))
    dw = torch.matmul(both.transpose(0, 1), v["x"])
    grads = [dx, *dw.split(case["n"])]
    return grads + list(both.sum(dim=0).split(case["n"])) if case["bias"] else grads
