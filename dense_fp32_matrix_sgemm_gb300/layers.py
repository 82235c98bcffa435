"""The operators around a transformer block's matrix products, for torch CUDA tensors.

``linear`` (bias, activation and residual in the product's epilogue), its
gradients ``linear_backward``, ``add_rmsnorm`` (residual addition and
root-mean-square norm, output in the input's type or as 8-bit rows with a
scale each), its gradients ``add_rmsnorm_backward``, and ``quantize_rows``.
Each call computes pointers and leading dimensions, allocates the outputs with
torch's allocator and enqueues the library's kernels (the C ABI of
include/sgemm_gb300_layers.h) on ``stream`` (default: torch's current stream;
outputs and scratch memory are allocated for the stream the call runs on).
Nothing synchronises.  Matrices are 2-D with a unit column stride and any row
stride; a weight may also be the transposed view of one.
"""
from __future__ import annotations

import functools

import torch

import dense_fp32_matrix_sgemm_gb300 as _sg

F32, BF16, F16, E4M3 = 0, 1, 2, 3
_TYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16, torch.float8_e4m3fn: E4M3}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_erf": 3, "silu": 4}


def _on_stream(fn):
    """Runs the call with its ``stream`` argument (a torch stream or a
    cudaStream_t as an int) current, so that torch's allocator hands out and
    takes back the call's memory in that stream's order."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kwargs):
        if stream is None:
            return fn(*args, **kwargs)
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=args[0].device)
        with torch.cuda.stream(stream):
            return fn(*args, **kwargs)
    return call


def _current(device):
    return torch.cuda.current_stream(device).cuda_stream


def _matrix(t, name, dtype=None, shape=None):
    """Leading dimension of a 2-D CUDA tensor with unit column stride."""
    if not t.is_cuda or t.dim() != 2 or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name} must be a 2-D CUDA tensor" + (f" of {dtype}" if dtype else ""))
    r, c = t.shape
    if shape is not None and (r, c) != shape:
        raise ValueError(f"{name} has shape {(r, c)}, expected {shape}")
    sr, sc = t.stride()
    if (sc != 1 and c > 1) or (sr < c and r > 1):
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return max(sr, c, 1) if r > 1 else max(c, 1)


def _vector(t, name, dtype, n):
    """Data pointer of a contiguous 1-D CUDA tensor of n elements, 0 for None."""
    if t is None:
        return 0
    if not t.is_cuda or t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or \
            (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of {n} elements")
    return t.data_ptr()


def _weight(w, name, k, dtype):
    """(out features, leading dimension, transW) of an (N, K) weight, stored
    by rows (transW = 1) or as the transposed view of a K x N matrix (0)."""
    if not w.is_cuda or w.dim() != 2 or w.dtype != dtype:
        raise TypeError(f"{name} must be a 2-D CUDA tensor of {dtype}")
    n, k2 = w.shape
    if k2 != k:
        raise ValueError(f"{name} has {k2} input features, expected {k}")
    sr, sc = w.stride()
    if sc == 1 and (sr >= k or n <= 1):
        return n, max(sr if n > 1 else k, k, 1), 1
    if sr == 1 and (sc >= n or k <= 1):
        return n, max(sc if k > 1 else n, n, 1), 0
    raise ValueError(f"{name} must have one unit stride")


def _scratch(workspace, need, device):
    if need == 0:
        return 0, 0, None
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return workspace.data_ptr(), workspace.numel(), workspace


def _type(t, name, allowed):
    code = _TYPES.get(t.dtype)
    if code is None or code not in allowed:
        raise TypeError(f"{name} has an unsupported type {t.dtype}")
    return code


def _activation(name):
    try:
        return ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}") from None


@_on_stream
def linear(x, weight, bias=None, *, activation="none", residual=None, x_scale=None, w_scale=None,
           out_dtype=None, save_preact=False, out=None, workspace=None):
    """act(x @ weight.T + bias) + residual, x (M, K), weight (N, K).

    float32 (FP32 accuracy), bfloat16, float16, or float8_e4m3fn with
    ``x_scale`` (M) and ``w_scale`` (N) float32 (as ``add_rmsnorm`` and
    ``quantize_rows`` make them) and a bfloat16 (default) or float16 result.
    bias, residual and out have the result's type; out may be residual.
    ``save_preact=True`` returns (y, z) with z the rounded pre-activation that
    ``linear_backward`` takes.  ``workspace``: a CUDA uint8 tensor, used where
    the call needs scratch memory and it is large enough."""
    dt = _type(x, "x", (F32, BF16, F16, E4M3))
    ldx = _matrix(x, "x")
    m, k = x.shape
    n, ldw, trans = _weight(weight, "weight", k, x.dtype)
    if dt == E4M3:
        out_dtype = out_dtype or torch.bfloat16
        if out_dtype not in (torch.bfloat16, torch.float16):
            raise TypeError("out_dtype must be bfloat16 or float16 for float8_e4m3fn operands")
        if x_scale is None or w_scale is None:
            raise ValueError("float8_e4m3fn operands need x_scale and w_scale")
        if not trans:
            raise ValueError("a float8_e4m3fn weight must be stored by rows")
    else:
        if out_dtype not in (None, x.dtype):
            raise TypeError("out_dtype is x's type")
        if x_scale is not None or w_scale is not None:
            raise ValueError("scales go with float8_e4m3fn operands only")
        out_dtype = x.dtype
    act = _activation(activation)
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=x.device)
        ldy = max(n, 1)
    else:
        ldy = _matrix(out, "out", out_dtype, (m, n))
    z, ldz = None, 0
    if save_preact:
        z = torch.empty((m, n), dtype=out_dtype, device=x.device)
        ldz = max(n, 1)
    ldr = _matrix(residual, "residual", out_dtype, (m, n)) if residual is not None else 0
    xp, wp = x.data_ptr(), weight.data_ptr()
    need = _sg.linear_workspace_size(dt, m, n, k, xp, ldx, wp, ldw, trans)
    ws, wsb, keep = _scratch(workspace, need, x.device)
    _sg.sgemm_linear(dt, m, n, k, xp, ldx, _vector(x_scale, "x_scale", torch.float32, m), wp, ldw,
                     trans, _vector(w_scale, "w_scale", torch.float32, n),
                     _vector(bias, "bias", out_dtype, n), act,
                     residual.data_ptr() if residual is not None else 0, ldr, _TYPES[out_dtype],
                     out.data_ptr(), ldy, z.data_ptr() if save_preact else 0, ldz, ws, wsb,
                     _current(x.device))
    return (out, z) if save_preact else out


@_on_stream
def linear_backward(dy, x, weight, preact=None, *, activation="none", need_dx=True, need_dw=True,
                    need_db=True, workspace=None):
    """Gradients (dx, dweight, dbias) of ``linear`` from dy (M, N), its x and
    weight, and the stored ``preact`` (not needed for activation "none");
    None where not asked for.  The residual's gradient is dy.  dweight has the
    weight's storage order.  float32, bfloat16 or float16."""
    dt = _type(dy, "dy", (F32, BF16, F16))
    lddy = _matrix(dy, "dy")
    m, n = dy.shape
    ldx = _matrix(x, "x", dy.dtype)
    k = x.shape[1]
    if x.shape[0] != m:
        raise ValueError(f"x has {x.shape[0]} rows, dy {m}")
    n2, ldw, trans = _weight(weight, "weight", k, dy.dtype)
    if n2 != n:
        raise ValueError(f"weight has {n2} output features, dy {n}")
    act = _activation(activation)
    if act and preact is None:
        raise ValueError("this activation's gradient needs preact")
    ldz = _matrix(preact, "preact", dy.dtype, (m, n)) if act else 0
    new = lambda *shape: torch.empty(shape, dtype=dy.dtype, device=dy.device)  # noqa: E731
    dx = new(m, k) if need_dx else None
    dw = (new(n, k) if trans else new(k, n).t()) if need_dw else None
    db = new(n) if need_db else None
    ptrs = dy.data_ptr(), x.data_ptr(), weight.data_ptr()
    need = _sg.linear_backward_workspace_size(dt, m, n, k, ptrs[0], lddy, act, ptrs[1], ldx,
                                              ptrs[2], ldw, trans)
    ws, wsb, keep = _scratch(workspace, need, dy.device)
    _sg.sgemm_linear_backward(dt, m, n, k, ptrs[0], lddy, preact.data_ptr() if act else 0, ldz, act,
                              ptrs[1], ldx, ptrs[2], ldw, trans,
                              dx.data_ptr() if need_dx else 0, max(k, 1),
                              dw.data_ptr() if need_dw else 0, max(k if trans else n, 1),
                              db.data_ptr() if need_db else 0, ws, wsb, _current(dy.device))
    return dx, dw, db


@_on_stream
def add_rmsnorm(x, weight, residual=None, *, eps=1e-6, quantize=False):
    """Root-mean-square norm of the rows of s = x + residual, times weight.

    Returns (y, s, rstd), or with ``quantize`` (q, scale, s, rstd): q
    float8_e4m3fn and scale float32 a row, y about q * scale[:, None].  Without
    a residual s is x itself.  x (rows, D) float32, bfloat16 or float16; rstd
    float32, for ``add_rmsnorm_backward``."""
    dt = _type(x, "x", (F32, BF16, F16))
    ldx = _matrix(x, "x")
    rows, d = x.shape
    wp = _vector(weight, "weight", x.dtype, d)
    s, sp, ldr, rp = x, 0, 0, 0
    if residual is not None:
        ldr = _matrix(residual, "residual", x.dtype, (rows, d))
        rp = residual.data_ptr()
        s = torch.empty((rows, d), dtype=x.dtype, device=x.device)
        sp = s.data_ptr()
    y = torch.empty((rows, d), dtype=torch.float8_e4m3fn if quantize else x.dtype, device=x.device)
    stats = torch.empty((2 if quantize else 1, rows), dtype=torch.float32, device=x.device)
    rstd = stats[0]
    scale = stats[1] if quantize else None
    ld = max(d, 1)
    _sg.sgemm_add_rmsnorm(dt, rows, d, x.data_ptr(), ldx, rp, ldr, wp, eps, sp, ld, y.data_ptr(),
                          ld, scale.data_ptr() if quantize else 0, rstd.data_ptr(),
                          _current(x.device))
    return (y, scale, s, rstd) if quantize else (y, s, rstd)


@_on_stream
def add_rmsnorm_backward(dy, s, rstd, weight, ds=None, *, need_dweight=True, workspace=None):
    """Gradients (dx, dweight) of ``add_rmsnorm`` from dy, the s and rstd it
    returned and the gradient ``ds`` that reaches s on the residual stream; dx
    is the gradient of x and of the residual alike."""
    dt = _type(dy, "dy", (F32, BF16, F16))
    lddy = _matrix(dy, "dy")
    rows, d = dy.shape
    lds = _matrix(s, "s", dy.dtype, (rows, d))
    ldds = _matrix(ds, "ds", dy.dtype, (rows, d)) if ds is not None else 0
    dx = torch.empty((rows, d), dtype=dy.dtype, device=dy.device)
    dw = torch.empty((d,), dtype=dy.dtype, device=dy.device) if need_dweight else None
    need = _sg.add_rmsnorm_backward_workspace_size(dt, rows, d) if need_dweight else 0
    ws, wsb, keep = _scratch(workspace, need, dy.device)
    _sg.sgemm_add_rmsnorm_backward(dt, rows, d, dy.data_ptr(), lddy, s.data_ptr(), lds,
                                   _vector(rstd, "rstd", torch.float32, rows),
                                   _vector(weight, "weight", dy.dtype, d),
                                   ds.data_ptr() if ds is not None else 0, ldds, dx.data_ptr(),
                                   max(d, 1), dw.data_ptr() if need_dweight else 0, ws, wsb,
                                   _current(dy.device))
    return dx, dw


@_on_stream
def quantize_rows(x):
    """(q, scale): the rows of x (float32, bfloat16 or float16) as
    float8_e4m3fn with one float32 scale each, x about q * scale[:, None]."""
    dt = _type(x, "x", (F32, BF16, F16))
    ldx = _matrix(x, "x")
    rows, d = x.shape
    q = torch.empty((rows, d), dtype=torch.float8_e4m3fn, device=x.device)
    scale = torch.empty((rows,), dtype=torch.float32, device=x.device)
    _sg.sgemm_quantize_rows(dt, rows, d, x.data_ptr(), ldx, q.data_ptr(), max(d, 1),
                            scale.data_ptr(), _current(x.device))
    return q, scale
