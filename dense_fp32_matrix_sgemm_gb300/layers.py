"""The operators around a transformer block's matrix products, for torch CUDA tensors.

``linear`` (bias, activation and residual in the product's epilogue), its
gradients ``linear_backward``, ``add_rmsnorm`` (residual addition and
root-mean-square norm, output in the input's type or as 8-bit rows with a
scale each), its gradients ``add_rmsnorm_backward``, and ``quantize_rows``.
Each call checks its tensors, allocates the outputs with torch's allocator and
enqueues the library's kernels (the C ABI of include/sgemm_gb300_layers.h) on
``stream`` (default: torch's current stream; outputs and scratch memory are
allocated for the stream the call runs on).  Nothing synchronises.  No gradient is
recorded: results of tensors that require one do not (the ``_backward`` functions
are the gradients, for a torch.autograd.Function or a training loop of one's own,
as examples/feed_forward.py has).  Matrices
are 2-D with a unit column stride and any row stride; a weight may also be the
transposed view of one.  All tensors of a call, its workspace and its stream are
of one device, and the call runs there whatever device is current.  The checks and the call itself are in ``_layers``, a
C++ extension built beside the library; there is no other route.
"""
from __future__ import annotations

import ctypes

import torch

import dense_fp32_matrix_sgemm_gb300 as _sg

_lib = _sg.load_library()
try:
    from . import _layers
except ImportError as e:
    raise _sg.SgemmUnavailable(
        f"the torch binding of the layer operators is not built or does not load ({e}); run "
        "__graft_entry__.build() or python -m dense_fp32_matrix_sgemm_gb300._build") from e
_layers.bind({name: ctypes.cast(getattr(_lib, name), ctypes.c_void_p).value
              for name in _sg.LAYER_ENTRIES}, _sg._check, torch.OutOfMemoryError)

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_erf": 3, "silu": 4}


def _activation(name):
    try:
        return ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}") from None


def _on(stream, like):
    """Context with ``stream`` (a torch stream or a cudaStream_t as an int)
    current: torch's allocator then hands out and takes back the call's memory
    in that stream's order."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    elif stream.device != like.device:
        raise ValueError(f"stream is of {stream.device}, the call's first tensor on {like.device}")
    return torch.cuda.stream(stream)


def linear(x, weight, bias=None, *, activation="none", residual=None, x_scale=None, w_scale=None,
           out_dtype=None, save_preact=False, out=None, workspace=None, stream=None):
    """act(x @ weight.T + bias) + residual, x (M, K), weight (N, K).

    float32 (FP32 accuracy; beyond 16 rows an infinity in x or weight may give NaN
    where the sum is infinite), bfloat16, float16, or float8_e4m3fn with
    ``x_scale`` (M) and ``w_scale`` (N) float32 (as ``add_rmsnorm`` and
    ``quantize_rows`` make them) and a bfloat16 (default) or float16 result.
    bias, residual and out have the result's type; out may be residual and overlaps
    nothing else that the call reads.
    ``save_preact=True`` returns (y, z) with z the rounded pre-activation that
    ``linear_backward`` takes.  ``workspace``: a CUDA uint8 tensor, used where
    the call needs scratch memory and it is large enough."""
    if stream is not None:
        with _on(stream, x):
            return linear(x, weight, bias, activation=activation, residual=residual,
                          x_scale=x_scale, w_scale=w_scale, out_dtype=out_dtype,
                          save_preact=save_preact, out=out, workspace=workspace)
    if out_dtype is not None and out_dtype != x.dtype and not (
            x.dtype == torch.float8_e4m3fn and out_dtype in (torch.bfloat16, torch.float16)):
        raise TypeError("out_dtype is x's type, or bfloat16 or float16 for float8_e4m3fn")
    return _layers.linear(x, weight, bias, _activation(activation), residual, x_scale, w_scale,
                          out_dtype is torch.float16, save_preact, out, workspace)


def linear_backward(dy, x, weight, preact=None, *, activation="none", need_dx=True, need_dw=True,
                    need_db=True, workspace=None, stream=None):
    """Gradients (dx, dweight, dbias) of ``linear`` from dy (M, N), its x and
    weight, and the stored ``preact`` (not needed for activation "none");
    None where not asked for.  The residual's gradient is dy.  dweight has the
    weight's storage order.  float32, bfloat16 or float16."""
    if stream is not None:
        with _on(stream, dy):
            return linear_backward(dy, x, weight, preact, activation=activation, need_dx=need_dx,
                                   need_dw=need_dw, need_db=need_db, workspace=workspace)
    return _layers.linear_backward(dy, x, weight, preact, _activation(activation), need_dx, need_dw,
                                   need_db, workspace)


def add_rmsnorm(x, weight, residual=None, *, eps=1e-6, quantize=False, stream=None):
    """Root-mean-square norm of the rows of s = x + residual, times weight.

    Returns (y, s, rstd), or with ``quantize`` (q, scale, s, rstd): q
    float8_e4m3fn and scale float32 a row, y about q * scale[:, None].  Without
    a residual s is x itself.  x (rows, D) float32, bfloat16 or float16; rstd
    float32, for ``add_rmsnorm_backward``.  Rows of no elements have the statistics
    of a row of zeros."""
    if stream is not None:
        with _on(stream, x):
            return add_rmsnorm(x, weight, residual, eps=eps, quantize=quantize)
    return _layers.add_rmsnorm(x, weight, residual, eps, quantize)


def add_rmsnorm_backward(dy, s, rstd, weight, ds=None, *, need_dweight=True, workspace=None,
                         stream=None):
    """Gradients (dx, dweight) of ``add_rmsnorm`` from dy, the s and rstd it
    returned and the gradient ``ds`` that reaches s on the residual stream; dx
    is the gradient of x and of the residual alike."""
    if stream is not None:
        with _on(stream, dy):
            return add_rmsnorm_backward(dy, s, rstd, weight, ds, need_dweight=need_dweight,
                                        workspace=workspace)
    return _layers.add_rmsnorm_backward(dy, s, rstd, weight, ds, need_dweight, workspace)


def quantize_rows(x, *, stream=None):
    """(q, scale): the rows of x (float32, bfloat16 or float16) as
    float8_e4m3fn with one float32 scale each, x about q * scale[:, None]."""
    if stream is not None:
        with _on(stream, x):
            return quantize_rows(x)
    return _layers.quantize_rows(x)
