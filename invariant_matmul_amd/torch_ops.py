"""Batch-invariant torch operators on top of the library.

The Tencent deterministic-inference article closes with vLLM's
batch-invariant mode, which replaces ``mm``, ``addmm``, ``matmul`` and
``linear`` with a GEMM whose configuration never depends on the batch size.
This module gives the same four operators on this library, and a context
manager that installs the library as torch's CUDA kernels of ``aten::mm`` and
``aten::addmm`` (through ``torch.library``, the mechanism of that mode), so
every CUDA product that reaches them takes the library's path:

    from invariant_matmul_amd import torch_ops
    y = torch_ops.linear(x, weight, bias)          # x [..., K], weight [N, K]
    with torch_ops.batch_invariant_mode():
        y = model(x)                               # nn.Linear, torch.mm, x.mm, @ ...

The split of K is planned from (N, K, dtype) alone (the library's rule) and
the single pass takes its output tile from M (GEMM_PLAN_TILE_BY_M), which
moves work between workgroups but never changes a bit, so row i of a result
depends only on row i of the input, on the weight and on K: never on how many
rows share the call.  A weight given as a transposed
view (``W.t()`` of a contiguous [N, K] tensor, which is how ``linear`` hands
it over) is read in place through the library's transposed-B plans.  Inputs
are fp16 or bf16 CUDA tensors; the result has the input dtype (fp32 sums,
one rounding at the end); a bias is added in fp32 before that rounding.

fp64 CUDA tensors go through the library's Ozaki-scheme product (int8
slices, default slice count and Fast Mode threshold: the Insight Edge cuTile
blog's FP64 emulation, here with one exponent per row, so it is batch-
invariant too); a bias is then added with one fp64 addition.  Any N and K.
Its domain: a row of the first operand or a column of the second that holds
a NaN or an infinity, a magnitude above 2^300, or only nonzero magnitudes
below 2^-300 gives NaN in its whole row or column of the result.

The direct functions raise for anything else.  Under the context manager the
library computes what it supports (2-D weights; fp16 / bf16 with N and K
multiples of 8, or fp64; alpha = beta = 1; a bias of N values); other CUDA
calls of aten::mm / aten::addmm (fp32 tensors, a full-matrix bias, other
alpha and beta) run on torch's own batched GEMM (aten::bmm, batch of one),
since the registration replaces torch's mm kernel while it is active.  CPU
tensors and batched products (aten::bmm) are not affected.  Autograd's
backward products go through aten::mm too, so they take the same path.

The operators around a linear layer keep the same promise, row by row:

    y, h = torch_ops.rms_norm(x, w, residual=r)        # h = x + r, y = norm(h) w
    q, s, h = torch_ops.rms_norm_quant(x, w, residual=r)  # fp8 rows and their scales

rms_norm takes part in autograd (its backward pass is a kernel of the library;
the weight's gradient is the one result that sums over rows).  The fp8 form
and quantize_rows are for serving: they refuse inputs that require a gradient.
"""
from __future__ import annotations

import contextlib
import functools
import threading
import warnings

import torch

from . import (PLAN_B_TRANSPOSED, PLAN_TILE_BY_M, gemm_plan_ex2, gemm_run, gemm_splitk_run,
               gemm_workspace_size, ozaki_plan, ozaki_run, ozaki_workspace_size, rms_norm_plan)
from . import quantize_rows as _quantize_rows
from . import rms_norm_backward as _rms_norm_backward
from . import rms_norm_run as _rms_norm_run

__all__ = ["mm", "addmm", "linear", "matmul", "batch_invariant_mode", "supported",
           "rms_norm", "rms_norm_forward", "rms_norm_backward", "rms_norm_quant", "quantize_rows"]

_DT = {torch.float16: "f16", torch.bfloat16: "bf16"}


@functools.lru_cache(maxsize=512)
def _plan(M: int, N: int, K: int, dt: str, flags: int):
    return gemm_plan_ex2(M, N, K, dt, dt, flags=flags)


def supported(a: torch.Tensor, b: torch.Tensor) -> bool:
    """True if a @ b (a [..., K], b [K, N]) is a product this module computes."""
    if not (a.is_cuda and b.is_cuda and b.dtype == a.dtype and b.dim() == 2 and a.dim() >= 1
            and a.shape[-1] == b.shape[0]):
        return False
    if a.dtype == torch.float64:
        return True
    return a.dtype in _DT and b.shape[0] % 8 == 0 and b.shape[1] % 8 == 0


@functools.lru_cache(maxsize=512)
def _ozaki_plan(M: int, N: int, K: int):
    return ozaki_plan(M, N, K, "i8")


def _product64(a2: torch.Tensor, b: torch.Tensor, bias) -> torch.Tensor:
    """a2 [M, K] @ b [K, N] (+ bias [N]) in fp64 by the Ozaki scheme."""
    M, K = a2.shape
    N = b.shape[1]
    out = torch.empty((M, N), dtype=torch.float64, device=a2.device)
    if M == 0 or N == 0:
        return out
    plan = _ozaki_plan(M, N, K)
    ws = torch.empty(max(1, ozaki_workspace_size(plan)), dtype=torch.uint8, device=a2.device)
    ozaki_run(plan, a2.contiguous(), b.contiguous(), out, ws)
    if bias is not None:
        out += bias.reshape(1, N).to(device=a2.device, dtype=torch.float64)
    return out


def _product(a2: torch.Tensor, b: torch.Tensor, bias) -> torch.Tensor:
    """a2 [M, K] @ b [K, N] (+ bias [N]) in the dtype of a2."""
    if a2.dtype == torch.float64:
        return _product64(a2, b, bias)
    M, K = a2.shape
    N = b.shape[1]
    dt = _DT[a2.dtype]
    a2 = a2.contiguous()
    flags = PLAN_TILE_BY_M
    if b.is_contiguous():
        bm = b
    elif b.t().is_contiguous():
        bm, flags = b.t(), flags | PLAN_B_TRANSPOSED  # the [N, K] weight itself
    else:
        bm = b.contiguous()
    out = torch.empty((M, N), dtype=a2.dtype, device=a2.device)
    if M == 0 or N == 0:
        return out
    bias32 = None
    if bias is not None:
        bias32 = bias.reshape(N).to(device=a2.device, dtype=torch.float32).contiguous()
    plan = _plan(M, N, K, dt, flags)
    if plan.info["split_k"] > 1:
        ws = torch.empty(max(1, gemm_workspace_size(plan) // 4), dtype=torch.float32,
                         device=a2.device)
        gemm_splitk_run(plan, a2, bm, out, ws, bias=bias32)
    else:
        gemm_run(plan, a2, bm, out, bias=bias32)
    return out


def _require(a, b):
    if not supported(a, b):
        raise ValueError(
            "invariant_matmul_amd.torch_ops: needs fp16/bf16 (K, N multiples of 8) or fp64 CUDA "
            "tensors, a [..., K] and a 2-D [K, N] second operand; got "
            f"{tuple(a.shape)} {a.dtype} @ "
            f"{tuple(b.shape)} {b.dtype}")


def mm(a: torch.Tensor, b: torch.Tensor) -> torch.Tensor:
    """a [M, K] @ b [K, N]."""
    if a.dim() != 2:
        raise ValueError("mm: a must be 2-D")
    _require(a, b)
    return _product(a, b, None)


def addmm(bias: torch.Tensor, a: torch.Tensor, b: torch.Tensor, *, beta=1, alpha=1) -> torch.Tensor:
    """bias + a @ b with a bias of N values (broadcast over rows); beta = alpha = 1."""
    if beta != 1 or alpha != 1:
        raise ValueError("addmm: only beta = alpha = 1")
    if a.dim() != 2:
        raise ValueError("addmm: a must be 2-D")
    _require(a, b)
    if bias.numel() != b.shape[1]:
        raise ValueError("addmm: the bias must hold N values")
    return _product(a, b, bias)


def linear(x: torch.Tensor, weight: torch.Tensor, bias=None) -> torch.Tensor:
    """x [..., K] @ weight[N, K]^T + bias."""
    wt = weight.t()
    _require(x, wt)
    lead = x.shape[:-1]
    y = _product(x.reshape(-1, x.shape[-1]), wt, bias)
    return y.reshape(*lead, weight.shape[0])


def matmul(a: torch.Tensor, b: torch.Tensor) -> torch.Tensor:
    """a [..., K] @ b [K, N] (leading dimensions of a are rows)."""
    _require(a, b)
    if a.dim() == 1:
        return _product(a.reshape(1, -1), b, None).reshape(b.shape[1])
    lead = a.shape[:-1]
    return _product(a.reshape(-1, a.shape[-1]), b, None).reshape(*lead, b.shape[1])


def _torch_mm(a: torch.Tensor, b: torch.Tensor) -> torch.Tensor:
    """a @ b on torch's batched GEMM (a batch of one); both operands contiguous."""
    return torch.bmm(a.unsqueeze(0).contiguous(), b.unsqueeze(0).contiguous()).squeeze(0)


def _row_bias(bias: torch.Tensor, N: int) -> bool:
    """True if bias holds N values broadcast over the rows."""
    return bias.numel() == N and (bias.dim() == 1 or (bias.dim() == 2 and bias.shape[0] == 1))


def _mode_mm(a, b):
    if a.dim() == 2 and supported(a, b):
        return _product(a, b, None)
    return _torch_mm(a, b)


def _mode_addmm(bias, a, b, *, beta=1, alpha=1):
    if (beta == 1 and alpha == 1 and a.dim() == 2 and supported(a, b)
            and _row_bias(bias, b.shape[1])):
        return _product(a, b, bias)
    r = _torch_mm(a, b)
    if alpha != 1:
        r = r * alpha
    if beta == 0:
        return r
    return r + (bias if beta == 1 else bias * beta)


# ---- Row norm and fp8 rows ------------------------------------------------------

_F8 = (torch.float8_e4m3fn, torch.float8_e5m2)


@functools.lru_cache(maxsize=512)
def _norm_plan(rows: int, cols: int, dtype, out_dtype, eps: float):
    return rms_norm_plan(rows, cols, dtype, out_dtype, eps)


def _dense(t: torch.Tensor) -> torch.Tensor:
    """t itself if the kernels can read it in place (contiguous, 16-byte
    aligned), else a copy."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _check_norm(where: str, x, weight, residual):
    if not (x.is_cuda and x.dtype in _DT and x.dim() >= 1 and x.shape[-1] % 8 == 0):
        raise ValueError(f"{where}: needs an fp16/bf16 CUDA tensor whose last size is a multiple "
                         f"of 8, got {tuple(x.shape)} {x.dtype} on {x.device}")
    if weight is not None and (weight.dtype != x.dtype or weight.device != x.device
                               or weight.shape != x.shape[-1:]):
        raise ValueError(f"{where}: weight must hold {x.shape[-1]} values of {x.dtype} on {x.device}")
    if residual is not None and (residual.dtype != x.dtype or residual.device != x.device
                                 or residual.shape != x.shape):
        raise ValueError(f"{where}: residual must have the shape, type and device of x")


def _refuse_grad(where: str, *tensors):
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise ValueError(f"{where} has no backward pass: call it under torch.no_grad() or with "
                         "detached tensors")


def _norm(x, weight, eps, residual, out_dtype, want_rstd):
    """(out, stream, row_scale or None, rstd or None), the outputs new tensors."""
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    out = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    h = x if residual is None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    lead = x.shape[:-1]
    scale = rstd = None
    if out_dtype in _F8:
        scale = torch.empty(lead, dtype=torch.float32, device=x.device)
    if want_rstd:
        rstd = torch.empty(lead, dtype=torch.float32, device=x.device)
    plan = _norm_plan(rows, cols, x.dtype, out_dtype, float(eps))
    if rows:
        x = _dense(x)
        if residual is None:
            h = x
        _rms_norm_run(plan, x, out, None if weight is None else _dense(weight),
                      None if residual is None else _dense(residual),
                      None if residual is None else h, scale, rstd)
    return out, h, scale, rstd


def rms_norm_forward(x: torch.Tensor, weight=None, eps: float = 1e-6, residual=None):
    """(y, h, rstd): the norm y of h = x + residual (h is x without a residual)
    and the fp32 reciprocal root mean square of each row of h, which
    rms_norm_backward takes.  No autograd: rms_norm is the differentiable form."""
    _check_norm("rms_norm_forward", x, weight, residual)
    y, h, _, rstd = _norm(x, weight, eps, residual, x.dtype, True)
    return y, h, rstd


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight, rstd: torch.Tensor, dh=None,
                      weight_grad: bool = True):
    """(dx, dweight) of rms_norm_forward: dy is the gradient of y, dh the gradient
    of h from its other uses (or None).  dx is the gradient of x and of the
    residual alike; dweight is None without a weight or with weight_grad=False."""
    _check_norm("rms_norm_backward", h, weight, dy)
    if dh is not None:
        _check_norm("rms_norm_backward", h, None, dh)
    if rstd.dtype != torch.float32 or rstd.shape != h.shape[:-1] or rstd.device != h.device:
        raise ValueError("rms_norm_backward: rstd must hold one float32 value per row of h")
    cols = h.shape[-1]
    rows = h.numel() // cols if cols else 0
    dx = torch.empty(h.shape, dtype=h.dtype, device=h.device)
    dw = ws = None
    plan = _norm_plan(rows, cols, h.dtype, h.dtype, 0.0)  # eps acts through rstd alone
    if weight is not None and weight_grad:
        dw = torch.empty(cols, dtype=h.dtype, device=h.device)
        if rows:
            ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=h.device)
    _rms_norm_backward(plan, _dense(dy), _dense(h), rstd.contiguous(), dx,
                       None if weight is None else _dense(weight),
                       None if dh is None else _dense(dh), dw, ws)
    return dx, dw


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h, _, rstd = _norm(x, weight, eps, residual, x.dtype, True)
        ctx.save_for_backward(h, weight, rstd)
        ctx.set_materialize_grads(False)
        return (y, h) if residual is not None else y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        need_x, need_w, need_r = ctx.needs_input_grad[:3]
        if dy is None:  # only the residual stream was used
            dw = torch.zeros_like(weight) if need_w and dh is not None else None
            return dh if need_x else None, dw, dh if need_r else None, None
        dx, dw = rms_norm_backward(dy, h, weight, rstd, dh, weight_grad=need_w)
        return dx if need_x else None, dw, dx if need_r else None, None


def rms_norm(x: torch.Tensor, weight=None, eps: float = 1e-6, residual=None):
    """y = h / sqrt(mean(h^2) + eps) * weight over the last dimension, with h = x.
    With a residual, h = x + residual, rounded to x's type, and the result is
    (y, h).  x, weight and residual are fp16 or bf16 of one type, the last
    size a multiple of 8 and at most 32768; statistics are fp32.  Row i of the
    result depends on row i alone.  Differentiable."""
    _check_norm("rms_norm", x, weight, residual)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad
                                       for t in (x, weight, residual)):
        return _RmsNorm.apply(x, weight, residual, eps)
    y, h, _, _ = _norm(x, weight, eps, residual, x.dtype, False)
    return (y, h) if residual is not None else y


def rms_norm_quant(x: torch.Tensor, weight=None, eps: float = 1e-6, residual=None,
                   dtype=torch.float8_e4m3fn):
    """(q, scale), or (q, scale, h) with a residual: rms_norm's rows before their
    rounding, as fp8 (e4m3fn or e5m2) rows with an fp32 scale each (the row is
    q * scale; the largest magnitude of a row becomes the type's largest
    value).  The last size is a multiple of 16."""
    _check_norm("rms_norm_quant", x, weight, residual)
    if dtype not in _F8 or x.shape[-1] % 16 != 0:
        raise ValueError("rms_norm_quant: dtype must be float8_e4m3fn or float8_e5m2 and the last "
                         "size a multiple of 16")
    _refuse_grad("rms_norm_quant", x, weight, residual)
    q, h, scale, _ = _norm(x, weight, eps, residual, dtype, False)
    return (q, scale, h) if residual is not None else (q, scale)


def quantize_rows(x: torch.Tensor, dtype=torch.float8_e4m3fn):
    """(q, scale): the rows of x (its last dimension) as fp8 with an fp32 scale
    each, for activations that no norm precedes and for weights [N, K]."""
    _check_norm("quantize_rows", x, None, None)
    if dtype not in _F8 or x.shape[-1] % 16 != 0:
        raise ValueError("quantize_rows: dtype must be float8_e4m3fn or float8_e5m2 and the last "
                         "size a multiple of 16")
    _refuse_grad("quantize_rows", x)
    cols = x.shape[-1]
    q = torch.empty(x.shape, dtype=dtype, device=x.device)
    scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    if x.numel():
        x2 = _dense(x).reshape(-1, cols)
        _quantize_rows(x2, q.reshape(-1, cols), scale.reshape(-1))
    return q, scale


_mode_lock = threading.Lock()
_mode_depth = 0
_mode_lib = None


@contextlib.contextmanager
def batch_invariant_mode():
    """Install this module's products as the CUDA kernels of aten::mm and
    aten::addmm while the context is active (nested contexts share one
    registration; the last exit removes it and torch's kernels return).  The
    registration is process-wide: products issued by other threads while it
    is active take the same path."""
    global _mode_depth, _mode_lib
    with _mode_lock:
        if _mode_depth == 0:
            lib = torch.library.Library("aten", "IMPL")
            with warnings.catch_warnings():
                # replacing a registered kernel is what this mode is for
                warnings.simplefilter("ignore")
                lib.impl("mm", _mode_mm, "CUDA")
                lib.impl("addmm", _mode_addmm, "CUDA")
            _mode_lib = lib
        _mode_depth += 1
    try:
        yield
    finally:
        with _mode_lock:
            _mode_depth -= 1
            if _mode_depth == 0:
                _mode_lib._destroy()
                _mode_lib = None
