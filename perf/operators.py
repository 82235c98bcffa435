"""The linear-layer operators on their working range: inputs, plain forms, the library's calls and exact values.

The operators are those around the matrix products of a pre-norm transformer block: the linear layer with bias,
activation and residual in its epilogue, its gradients, the root-mean-square norm with the residual's addition (its
output in the input's type or in 8 bits with a scale a row), its gradients, and the row quantiser that makes 8-bit
weights and activations.  ``run`` computes an operator in elementary torch operations in 32 bits, or, with ``own``
set, through the calls that a user makes of the library.
"""
import math

import torch

own = False

EPS = 1e-6            # the norm's epsilon
E4M3_MAX = 448.0      # largest finite value of the 8-bit type
AMAX_FLOOR = 1e-30    # a row of zeros gets the scale AMAX_FLOOR / E4M3_MAX

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_erf", "silu")


def _linear(name, dtype, m, n, k, act="none", bias=False, residual=False, preact=False, w_kn=False):
    return {"name": name, "op": "linear", "dtype": dtype, "m": m, "n": n, "k": k, "act": act, "bias": bias,
            "residual": residual, "preact": preact, "w_kn": w_kn}


def listed():
    return [
        # one token of a decoding step through a gate projection: every weight is read once, latency counts
        _linear("linear_token_bf16", "bf16", 1, 4096, 4096, act="silu", bias=True),
        # a training step's up-projection, which keeps the pre-activation for its gradient
        _linear("linear_train_bf16", "bf16", 4096, 8192, 4096, act="gelu", bias=True, preact=True),
        # full-precision layer of ragged sizes: neither rows nor columns a multiple of any tile or vector
        _linear("linear_ragged_f32", "f32", 2049, 3071, 1537, act="relu", bias=True, residual=True),
        # prefill through a down-projection on 8-bit weights and activations, added to the residual stream
        _linear("linear_prefill_e4m3", "e4m3", 8192, 8192, 8192, residual=True),
        # gradients of the training up-projection
        {"name": "linear_backward_bf16", "op": "linear_backward", "dtype": "bf16", "m": 4096, "n": 8192, "k": 4096,
         "act": "gelu", "bias": True, "w_kn": False},
        # gradients of a small full-precision head of odd sizes
        {"name": "linear_backward_ragged_f32", "op": "linear_backward", "dtype": "f32", "m": 500, "n": 777, "k": 1001,
         "act": "silu", "bias": True, "w_kn": False},
        # the norm before a projection in a decoding step, written as the 8-bit row that the product reads
        {"name": "add_rmsnorm_token_e4m3", "op": "add_rmsnorm", "dtype": "bf16", "rows": 1, "d": 4096,
         "residual": True, "quantize": True},
        # the norm of a prefill or a training step
        {"name": "add_rmsnorm_prefill_bf16", "op": "add_rmsnorm", "dtype": "bf16", "rows": 8192, "d": 8192,
         "residual": True, "quantize": False},
        # its gradient in a training step, joined with the residual stream's
        {"name": "add_rmsnorm_backward_bf16", "op": "add_rmsnorm_backward", "dtype": "bf16", "rows": 8192, "d": 4096,
         "stream_grad": True},
        # the same of an odd width in full precision, with few rows to sum the weight's gradient over
        {"name": "add_rmsnorm_backward_odd_f32", "op": "add_rmsnorm_backward", "dtype": "f32", "rows": 1000, "d": 1001,
         "stream_grad": False},
        # the activations of a decoding batch between two 8-bit products
        {"name": "quantize_rows_batch_bf16", "op": "quantize_rows", "dtype": "bf16", "rows": 64, "d": 8192},
        # a weight matrix brought to 8 bits
        {"name": "quantize_rows_weight_bf16", "op": "quantize_rows", "dtype": "bf16", "rows": 8192, "d": 8192},
    ]


def _size(rng, low, high):
    """Log-uniform; often a multiple of 64 where it is large enough, as widths are, else any number."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if v >= 128 and rng.random() < 0.6:
        v = v // 64 * 64
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "add_rmsnorm", "add_rmsnorm_backward", "quantize_rows"])
    if op == "linear":
        c = _linear("", rng.choice(["f32", "bf16", "bf16", "f16", "e4m3"]), _size(rng, 1, 8192), _size(rng, 16, 8192),
                    _size(rng, 16, 8192), act=rng.choice(ACTIVATIONS), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5, preact=rng.random() < 0.3)
        c["w_kn"] = c["dtype"] != "e4m3" and rng.random() < 0.3
        del c["name"]
        return c
    if op == "linear_backward":
        return {"op": op, "dtype": rng.choice(["f32", "bf16", "bf16", "f16"]), "m": _size(rng, 1, 8192),
                "n": _size(rng, 16, 8192), "k": _size(rng, 16, 4096), "act": rng.choice(ACTIVATIONS),
                "bias": rng.random() < 0.7, "w_kn": rng.random() < 0.3}
    c = {"op": op, "dtype": rng.choice(["f32", "bf16", "bf16", "f16"]), "rows": _size(rng, 1, 16384),
         "d": _size(rng, 16, 8192)}
    if op == "add_rmsnorm":
        c |= {"residual": rng.random() < 0.7, "quantize": rng.random() < 0.4}
    elif op == "add_rmsnorm_backward":
        c |= {"stream_grad": rng.random() < 0.7}
    return c


# ---------------------------------------------------------------------------------------------------- inputs


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def _activations(g, rows, d):
    """Unit-variance rows of different size, with a few columns far larger than the others, as hidden states have."""
    x = _normal(g, rows, d)
    x *= torch.exp(_normal(g, rows, 1, std=0.3))
    big = torch.randint(0, d, (max(1, d // 512),), generator=g, device="cuda")
    x[:, big] *= 12.0
    return x


def _to_e4m3(x):
    a = x.abs().amax(1).clamp_min(AMAX_FLOOR)
    q = (x * (E4M3_MAX / a)[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q, a / E4M3_MAX


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    if case["op"] in ("linear", "linear_backward"):
        m, n, k = case["m"], case["n"], case["k"]
        out = DTYPES["bf16" if case["dtype"] == "e4m3" else case["dtype"]]
        w = _normal(g, n, k, std=k ** -0.5)
        if case["dtype"] == "e4m3":
            s["x"], s["x_scale"] = _to_e4m3(_activations(g, m, k))
            s["w"], s["w_scale"] = _to_e4m3(w)
        else:
            s["x"] = (_activations(g, m, k) if case["op"] == "linear" else _normal(g, m, k)).to(out)
            # a weight stored with the outputs contiguous is the transposed view of a K x N matrix
            s["w"] = w.to(out).t().contiguous().t() if case["w_kn"] else w.to(out)
            s["x_scale"] = s["w_scale"] = None
        s["b"] = _normal(g, n, std=0.2).to(out) if case["bias"] else None
        if case["op"] == "linear":
            s["r"] = _activations(g, m, n).to(out) if case["residual"] else None
        else:
            s["z"] = None if case["act"] == "none" else _normal(g, m, n).to(out)
            s["dy"] = _normal(g, m, n).to(out)
        s["out"] = out
        return s
    rows, d, t = case["rows"], case["d"], DTYPES[case["dtype"]]
    s["x"] = _activations(g, rows, d).to(t)
    if case["op"] == "quantize_rows":
        return s
    s["w"] = (1.0 + _normal(g, d, std=0.1)).to(t)
    if case["op"] == "add_rmsnorm":
        s["r"] = _activations(g, rows, d).to(t) if case["residual"] else None
    else:
        s["dy"] = _normal(g, rows, d).to(t)
        s["ds"] = _normal(g, rows, d).to(t) if case["stream_grad"] else None
        s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
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
    p = 1.0 / (1.0 + torch.exp(-z))
    return p * (1.0 + z * (1.0 - p))


def _plain(s):
    if s["op"] == "linear":
        x, w = s["x"].float(), s["w"].float()
        if s["x_scale"] is not None:
            x, w = x * s["x_scale"][:, None], w * s["w_scale"][:, None]
        z = x @ w.t()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(z, s["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        y = y.to(s["out"])
        return (y, z.to(s["out"])) if s["preact"] else y
    if s["op"] == "linear_backward":
        dz = s["dy"].float()
        if s["z"] is not None:
            dz = dz * _act_grad(s["z"].float(), s["act"])
        dx = (dz @ s["w"].float()).to(s["out"])
        dw = (dz.t() @ s["x"].float()).to(s["out"])
        return (dx, dw, dz.sum(0).to(s["out"])) if s["bias"] else (dx, dw)
    if s["op"] == "quantize_rows":
        return _to_e4m3(s["x"].float())
    if s["op"] == "add_rmsnorm":
        h = s["x"].float()
        if s["r"] is not None:
            h = h + s["r"].float()
        rstd = torch.rsqrt(h.square().mean(1) + EPS)
        y = h * rstd[:, None] * s["w"].float()
        h = h.to(s["x"].dtype)
        return (*_to_e4m3(y), h, rstd) if s["quantize"] else (y.to(s["x"].dtype), h, rstd)
    h, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    g = dy * s["w"].float()
    dx = rstd * (g - h * rstd.square() * (g * h).mean(1, keepdim=True))
    if s["ds"] is not None:
        dx = dx + s["ds"].float()
    return dx.to(s["x"].dtype), (dy * h * rstd).sum(0).to(s["x"].dtype)


def run(state):
    s = state
    if not own:
        return _plain(s)
    import dense_fp32_matrix_sgemm_gb300 as sg
    if s["op"] == "linear":
        return sg.linear(s["x"], s["w"], s["b"], activation=s["act"], residual=s["r"], x_scale=s["x_scale"],
                         w_scale=s["w_scale"], save_preact=s["preact"])
    if s["op"] == "linear_backward":
        dx, dw, db = sg.linear_backward(s["dy"], s["x"], s["w"], s["z"], activation=s["act"], need_db=s["bias"])
        return (dx, dw, db) if s["bias"] else (dx, dw)
    if s["op"] == "quantize_rows":
        return sg.quantize_rows(s["x"])
    if s["op"] == "add_rmsnorm":
        return sg.add_rmsnorm(s["x"], s["w"], s["r"], eps=EPS, quantize=s["quantize"])
    return sg.add_rmsnorm_backward(s["dy"], s["x"], s["rstd"], s["w"], s["ds"])


# ---------------------------------------------------------------------------------------------------- cost and exact values


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        o = 2 if case["dtype"] == "e4m3" else e
        scales = 4 * (m + n) if case["dtype"] == "e4m3" else 0
        moved = e * (m * k + n * k) + scales + o * m * n * (1 + case["residual"] + case["preact"]) + o * n * case["bias"]
        return {"bytes": moved, "flops": 2 * m * n * k}
    if case["op"] == "linear_backward":
        m, n, k = case["m"], case["n"], case["k"]
        moved = e * (2 * m * k + 2 * n * k + m * n * (1 + (case["act"] != "none")) + n * case["bias"])
        return {"bytes": moved, "flops": 4 * m * n * k}
    r, d = case["rows"], case["d"]
    if case["op"] == "quantize_rows":
        return {"bytes": r * d * (e + 1) + 4 * r, "flops": 3 * r * d}
    if case["op"] == "add_rmsnorm":
        stream = 2 * e if case["residual"] else 0      # the residual read and the sum written
        y = r * d + 4 * r if case["quantize"] else r * d * e
        return {"bytes": r * d * (e + stream) + y + e * d + 4 * r, "flops": (5 + 3 * case["quantize"]) * r * d}
    return {"bytes": r * d * e * (3 + case["stream_grad"]) + 2 * e * d + 4 * r, "flops": 9 * r * d}


def exact(case, seed):
    """The same outputs in 64 bits, not rounded to the output's type (8-bit codes: the quotients they round)."""
    s = prepare(case, seed)
    v = {k: t.to(torch.float64) for k, t in s.items() if isinstance(t, torch.Tensor)}
    if case["op"] == "quantize_rows":
        top = v["x"].abs().max(dim=1).values.clamp(min=AMAX_FLOOR)
        return v["x"] / top.unsqueeze(1) * E4M3_MAX, top / E4M3_MAX
    if case["op"] == "add_rmsnorm":
        h = v["x"] + v["r"] if case["residual"] else v["x"]
        inv = 1.0 / torch.sqrt((h * h).sum(dim=1) / h.shape[1] + EPS)
        y = torch.einsum("rd,r,d->rd", h, inv, v["w"])
        if not case["quantize"]:
            return y, h, inv
        top = y.abs().max(dim=1).values.clamp(min=AMAX_FLOOR)
        return y / top.unsqueeze(1) * E4M3_MAX, top / E4M3_MAX, h, inv
    if case["op"] == "add_rmsnorm_backward":
        n = v["x"] * v["rstd"].unsqueeze(1)             # the normalised rows
        g = v["dy"] * v["w"]
        dx = (g - n * (g * n).sum(dim=1, keepdim=True) / n.shape[1]) * v["rstd"].unsqueeze(1)
        if case["stream_grad"]:
            dx = dx + v["ds"]
        return dx, torch.einsum("rd,rd->d", v["dy"], n)

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

    if case["op"] == "linear":
        z = torch.matmul(v["x"], v["w"].transpose(0, 1))
        if "x_scale" in v:
            z = z * v["x_scale"].unsqueeze(1) * v["w_scale"]
        if case["bias"]:
            z = z + v["b"]
        y = slope_and_value(z)[1]
        y = y + v["r"] if case["residual"] else y
        return (y, z) if case["preact"] else y
    dz = v["dy"] * slope_and_value(v["z"])[0] if "z" in v else v["dy"]
    grads = (torch.matmul(dz, v["w"]), torch.matmul(dz.transpose(0, 1), v["x"]))
    return (*grads, dz.sum(dim=0)) if case["bias"] else grads
