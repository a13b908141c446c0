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
the weight's gradient is the one result that sums over rows).  The others are
for serving and refuse inputs that require a gradient.  None has a derivative in
forward mode: all refuse dual tensors.

    wq, ws = torch_ops.quantize_rows(W)                # once
    y = torch_ops.linear_f8(q, s, wq, ws)              # fp8 rows and their scales
    w4 = torch_ops.pack_w4(q4, scales, zeros)          # once
    y = torch_ops.linear_w4(x, w4, bias)               # 4-bit weights
"""
from __future__ import annotations

import contextlib
import functools
import math
import threading
import warnings

import torch
from torch.autograd import forward_ad

from . import (PLAN_B_TRANSPOSED, PLAN_FP8_FP32_ACCUM, PLAN_TILE_BY_M, GemmError, _dtype_code,
               gemm_plan_ex2, gemm_run, gemm_splitk_run, gemm_workspace_size, lib, ozaki_plan,
               ozaki_run, ozaki_workspace_size, rms_norm_plan, w4_packed_size, w4_plan)

__all__ = ["mm", "addmm", "linear", "matmul", "batch_invariant_mode", "supported",
           "rms_norm", "rms_norm_forward", "rms_norm_backward", "rms_norm_quant", "quantize_rows",
           "linear_f8", "W4Weight", "pack_w4", "linear_w4"]

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


# ---- Row norm, fp8 rows, 4-bit weights --------------------------------------------
#
# These operators check their tensors here and hand addresses straight to the
# C ABI (which checks the memory behind them): a decode step calls them with a
# few microseconds of GPU work each, where a second round of checks would cost
# more than the kernel.

_F8 = (torch.float8_e4m3fn, torch.float8_e5m2)


@functools.lru_cache(maxsize=512)
def _norm_plan(rows: int, cols: int, dtype, out_dtype, eps: float):
    return rms_norm_plan(rows, cols, dtype, out_dtype, eps)


@functools.lru_cache(maxsize=512)
def _f8_plan(M: int, N: int, K: int, dtype, out_dtype, flags: int):
    # one pass, never a split of K: its bits are those of every M, and a split
    # workspace [split, M, N] would cost a long batch more than the product
    return gemm_plan_ex2(M, N, K, dtype, out_dtype, split_k=1, flags=flags)


@functools.lru_cache(maxsize=512)
def _w4_plan(M: int, N: int, K: int, dtype, group: int):
    return w4_plan(M, N, K, dtype, group)


def _dense(t: torch.Tensor) -> torch.Tensor:
    """t itself if the kernels can read it in place (contiguous, 16-byte
    aligned), else a copy."""
    if not t.is_contiguous():
        return t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _per_row(shape, device) -> torch.Tensor:
    """A new fp32 tensor with a value per row of `shape` (sizes given one by one
    take torch half the time of a tuple)."""
    if len(shape) == 2:
        return torch.empty(shape[0], dtype=torch.float32, device=device)
    return torch.empty(shape[:-1], dtype=torch.float32, device=device)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _stream_of(where: str, device) -> int:
    """The current stream of the current device, which must be the tensors'."""
    index = device.index
    if index != torch._C._cuda_getDevice():
        raise ValueError(f"{where}: the tensors are on {device}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(index)


def _done(status: int, where: str):
    if status:
        raise GemmError(status, where)


def _refuse_grad(where: str, *tensors):
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise ValueError(f"{where} has no backward pass: call it under torch.no_grad() or with "
                         "detached tensors")
    _refuse_tangent(where, *tensors)


def _refuse_tangent(where: str, *tensors):
    """Dual tensors of torch.autograd.forward_ad hold a tangent that requires_grad does not
    show (nor does torch.no_grad() stop it), and that a new tensor would not have."""
    if forward_ad._current_level >= 0 and any(  # inside a dual_level()
            t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise ValueError(f"{where} has no forward-mode derivative: call it with the primals of dual tensors")


def _check_norm(where: str, x, weight, residual):
    shape, dtype, device = x.shape, x.dtype, x.device
    if not (x.is_cuda and dtype in _DT and shape and shape[-1] % 8 == 0):
        raise ValueError(f"{where}: needs an fp16/bf16 CUDA tensor whose last size is a multiple "
                         f"of 8, got {tuple(shape)} {dtype} on {device}")
    if weight is not None and (weight.dtype != dtype or weight.device != device
                               or weight.shape != shape[-1:]):
        raise ValueError(f"{where}: weight must hold {shape[-1]} values of {dtype} on {device}")
    if residual is not None and (residual.dtype != dtype or residual.device != device
                                 or residual.shape != shape):
        raise ValueError(f"{where}: residual must have the shape, type and device of x")


def _check_f8_rows(where: str, x, dtype):
    if dtype not in _F8 or x.shape[-1] % 16 != 0:
        raise ValueError(f"{where}: dtype must be float8_e4m3fn or float8_e5m2 and the last size a "
                         "multiple of 16")


def _norm(where, x, weight, eps, residual, out_dtype, want_rstd):
    """(out, stream, row_scale or None, rstd or None), the outputs new tensors."""
    shape, device = x.shape, x.device
    stream = _stream_of(where, device)
    cols = shape[-1]
    rows = x.numel() // cols if cols else math.prod(shape[:-1])
    plan = _norm_plan(rows, cols, x.dtype, out_dtype, eps)
    x = _dense(x)
    out = torch.empty_like(x, dtype=out_dtype)
    h, scale, rstd = x, None, None
    w_at = r_at = h_at = scale_at = rstd_at = 0
    if residual is not None:
        h = torch.empty_like(x)
        residual = _dense(residual)
        r_at, h_at = residual.data_ptr(), h.data_ptr()
    if weight is not None:
        weight = _dense(weight)
        w_at = weight.data_ptr()
    if out_dtype in _F8:
        scale = _per_row(shape, device)
        scale_at = scale.data_ptr()
    if want_rstd:
        rstd = _per_row(shape, device)
        rstd_at = rstd.data_ptr()
    if rows:
        status = lib().rms_norm_run(plan.handle, x.data_ptr(), r_at, w_at, out.data_ptr(), scale_at,
                                    h_at, rstd_at, stream)
        if status:
            raise GemmError(status, where)
    return out, h, scale, rstd


def rms_norm_forward(x: torch.Tensor, weight=None, eps: float = 1e-6, residual=None):
    """(y, h, rstd): the norm y of h = x + residual (h is x without a residual)
    and the fp32 reciprocal root mean square of each row of h, which
    rms_norm_backward takes.  No autograd: rms_norm is the differentiable form."""
    _check_norm("rms_norm_forward", x, weight, residual)
    _refuse_tangent("rms_norm_forward", x, weight, residual)
    y, h, _, rstd = _norm("rms_norm_forward", x, weight, eps, residual, x.dtype, True)
    return y, h, rstd


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight, rstd: torch.Tensor, dh=None,
                      weight_grad: bool = True):
    """(dx, dweight) of rms_norm_forward: dy is the gradient of y, dh the gradient
    of h from its other uses (or None).  dx is the gradient of x and of the
    residual alike; dweight is None without a weight or with weight_grad=False."""
    where = "rms_norm_backward"
    _check_norm(where, h, weight, dy)
    shape, device = h.shape, h.device
    if dh is not None and (dh.dtype != h.dtype or dh.device != device or dh.shape != shape):
        raise ValueError("rms_norm_backward: dh must have the shape, type and device of h")
    if rstd.dtype != torch.float32 or rstd.shape != shape[:-1] or rstd.device != device:
        raise ValueError("rms_norm_backward: rstd must hold one float32 value per row of h")
    _refuse_tangent(where, dy, h, weight, rstd, dh)
    stream = _stream_of(where, device)
    cols = shape[-1]
    rows = h.numel() // cols if cols else 0
    plan = _norm_plan(rows, cols, h.dtype, h.dtype, 0.0)  # eps acts through rstd alone
    dy, h, rstd = _dense(dy), _dense(h), rstd.contiguous()
    dx = torch.empty_like(h)
    dw = ws = None
    nws = 0
    if weight is not None:
        weight = _dense(weight)
        if weight_grad:
            dw = torch.empty_like(weight)
            nws = plan.workspace_bytes
            ws = torch.empty(nws, dtype=torch.uint8, device=device)
    if dh is not None:
        dh = _dense(dh)
    _done(lib().rms_norm_backward(plan.handle, dy.data_ptr(), h.data_ptr(), _ptr(weight),
                                  rstd.data_ptr(), _ptr(dh), dx.data_ptr(), _ptr(dw), _ptr(ws), nws,
                                  stream), where)
    return dx, dw


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h, _, rstd = _norm("rms_norm", x, weight, eps, residual, x.dtype, True)
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
    result depends on row i alone.  Differentiable in reverse mode, once (dual
    tensors of torch.autograd.forward_ad are refused)."""
    _check_norm("rms_norm", x, weight, residual)
    _refuse_tangent("rms_norm", x, weight, residual)
    if torch.is_grad_enabled() and (x.requires_grad or (weight is not None and weight.requires_grad)
                                    or (residual is not None and residual.requires_grad)):
        return _RmsNorm.apply(x, weight, residual, eps)
    y, h, _, _ = _norm("rms_norm", x, weight, eps, residual, x.dtype, False)
    return (y, h) if residual is not None else y


def rms_norm_quant(x: torch.Tensor, weight=None, eps: float = 1e-6, residual=None,
                   dtype=torch.float8_e4m3fn):
    """(q, scale), or (q, scale, h) with a residual: rms_norm's rows before their
    rounding, as fp8 (e4m3fn or e5m2) rows with an fp32 scale each (the row is
    q * scale; the largest magnitude of a row becomes the type's largest
    value).  The last size is a multiple of 16."""
    where = "rms_norm_quant"
    _check_norm(where, x, weight, residual)
    _check_f8_rows(where, x, dtype)
    _refuse_grad(where, x, weight, residual)
    q, h, scale, _ = _norm(where, x, weight, eps, residual, dtype, False)
    return (q, scale, h) if residual is not None else (q, scale)


def quantize_rows(x: torch.Tensor, dtype=torch.float8_e4m3fn):
    """(q, scale): the rows of x (its last dimension) as fp8 with an fp32 scale
    each, for activations that no norm precedes and for weights [N, K]."""
    where = "quantize_rows"
    _check_norm(where, x, None, None)
    _check_f8_rows(where, x, dtype)
    _refuse_grad(where, x)
    stream = _stream_of(where, x.device)
    x = _dense(x)
    q = torch.empty_like(x, dtype=dtype)
    scale = _per_row(x.shape, x.device)
    rows = scale.numel()
    if rows:
        _done(lib().quantize_rows(rows, x.shape[-1], _dtype_code(x.dtype), _dtype_code(dtype),
                                  x.data_ptr(), q.data_ptr(), scale.data_ptr(), stream), where)
    return q, scale


def _bias32(where: str, bias, N: int, device):
    if bias is None:
        return None
    if bias.numel() != N or bias.device != device:
        raise ValueError(f"{where}: the bias must hold {N} values on {device}")
    return bias.reshape(N).to(torch.float32).contiguous()


def linear_f8(x: torch.Tensor, x_scale: torch.Tensor, weight: torch.Tensor,
              weight_scale: torch.Tensor, bias=None, out_dtype=torch.bfloat16,
              fp32_accum: bool = False) -> torch.Tensor:
    """y = (x x_scale) @ (weight weight_scale)^T + bias for fp8 rows with scales.

    x [..., K] and weight [N, K] are float8_e4m3fn or float8_e5m2 (both the
    same; K and N multiples of 16), x_scale fp32 [...] (one per row) and
    weight_scale fp32 [N], as rms_norm_quant and quantize_rows leave them.
    The products are summed on the fp8 matrix step (8 neighbours in a window of 13
    binades, then fp32), scaled by row and by
    column in fp32, the bias added in fp32, and the result rounded once to
    out_dtype (bf16, fp16 or fp32).  fp32_accum=True sums on the fp16 step
    instead (half the matrix rate, no kernel of few rows; the fp32 error bound for
    every K).  Row i of
    y depends on row i of x, its scale and the weight alone."""
    where = "linear_f8"
    dev = x.device
    if not (x.is_cuda and x.dtype in _F8 and x.dim() >= 1 and weight.dim() == 2
            and weight.dtype == x.dtype and weight.device == dev
            and weight.shape[1] == x.shape[-1]
            and weight.shape[0] % 16 == 0 and weight.shape[1] % 16 == 0):
        raise ValueError(
            "linear_f8: needs fp8 CUDA tensors of one type, x [..., K] and weight [N, K] with K and "
            f"N multiples of 16; got {tuple(x.shape)} {x.dtype} on {x.device} and "
            f"{tuple(weight.shape)} {weight.dtype} on {weight.device}")
    if out_dtype not in (torch.bfloat16, torch.float16, torch.float32):
        raise ValueError("linear_f8: out_dtype must be bfloat16, float16 or float32")
    N, K = weight.shape
    lead = x.shape[:-1]
    if not (x_scale.dtype == weight_scale.dtype == torch.float32 and x_scale.shape == lead
            and weight_scale.shape == (N,) and x_scale.device == weight_scale.device == dev):
        raise ValueError(
            f"linear_f8: x_scale must be float32 {tuple(lead)} and weight_scale float32 {(N,)} on "
            f"{dev}; got {x_scale.dtype} {tuple(x_scale.shape)} on {x_scale.device} and "
            f"{weight_scale.dtype} {tuple(weight_scale.shape)} on {weight_scale.device}")
    bias = _bias32(where, bias, N, dev)
    _refuse_grad(where, x, x_scale, weight, weight_scale, bias)
    stream = _stream_of(where, dev)
    M = x_scale.numel()
    out = torch.empty(*lead, N, dtype=out_dtype, device=dev)
    if M == 0 or N == 0:
        return out
    x, weight = _dense(x), _dense(weight)
    x_scale, weight_scale = x_scale.contiguous(), weight_scale.contiguous()
    flags = PLAN_TILE_BY_M | PLAN_B_TRANSPOSED | (PLAN_FP8_FP32_ACCUM if fp32_accum else 0)
    plan = _f8_plan(M, N, K, x.dtype, out_dtype, flags)
    _done(lib().gemm_run_scaled(plan.handle, x.data_ptr(), weight.data_ptr(), x_scale.data_ptr(),
                                weight_scale.data_ptr(), _ptr(bias), out.data_ptr(), stream), where)
    return out


class W4Weight:
    """A 4-bit weight [N, K] as linear_w4 reads it: made by pack_w4, or again from its
    packed bytes (a contiguous uint8 vector, as pack_w4 left it) and sizes."""

    __slots__ = ("packed", "N", "K", "group", "dtype")

    def __init__(self, packed: torch.Tensor, N: int, K: int, group: int, dtype: torch.dtype):
        # linear_w4 reads by the sizes: fewer bytes would be read past their end
        size = w4_packed_size(_w4_plan(1, N, K, dtype, group))
        if packed.dtype != torch.uint8 or packed.shape != (size,) or not packed.is_contiguous():
            raise ValueError(f"W4Weight: [{N}, {K}] in groups of {group} is a contiguous uint8 vector of {size} "
                             f"bytes, got {tuple(packed.shape)} {packed.dtype}")
        self.packed, self.N, self.K, self.group, self.dtype = packed, N, K, group, dtype

    def to(self, device) -> "W4Weight":
        return W4Weight(self.packed.to(device), self.N, self.K, self.group, self.dtype)


def pack_w4(q: torch.Tensor, scales: torch.Tensor, zeros=None) -> W4Weight:
    """Lay out a 4-bit weight once, for linear_w4.

    q: uint8 [N, K / 2], byte j of a row holding element 2 j in its low and
    2 j + 1 in its high half; scales [N, K / group], fp16 or bf16 (the type of
    the activations), group 32, 64 or 128; zeros: uint8 [N, K / group], or None
    for 8.  The weight is scales (q - zeros).  N is a multiple of 8."""
    where = "pack_w4"
    if not (q.is_cuda and q.dtype == torch.uint8 and q.dim() == 2 and scales.dim() == 2
            and scales.dtype in _DT and scales.device == q.device and scales.shape[0] == q.shape[0]):
        raise ValueError("pack_w4: needs uint8 q [N, K / 2] and fp16/bf16 scales [N, K / group] on one "
                         f"CUDA device; got {tuple(q.shape)} {q.dtype} on {q.device} and "
                         f"{tuple(scales.shape)} {scales.dtype} on {scales.device}")
    N, K = q.shape[0], 2 * q.shape[1]
    groups = scales.shape[1]
    group = K // groups if groups else 0
    if N % 8 != 0 or group not in (32, 64, 128) or groups * group != K:
        raise ValueError(f"pack_w4: N = {N} must be a multiple of 8 and K = {K} hold {groups} groups "
                         "of 32, 64 or 128")
    if zeros is not None and (zeros.dtype != torch.uint8 or zeros.shape != scales.shape
                              or zeros.device != q.device):
        raise ValueError("pack_w4: zeros must be uint8 of the shape and device of scales")
    _refuse_grad(where, scales)
    stream = _stream_of(where, q.device)
    plan = _w4_plan(1, N, K, scales.dtype, group)
    packed = torch.empty(w4_packed_size(plan), dtype=torch.uint8, device=q.device)
    q, scales = q.contiguous(), scales.contiguous()
    if zeros is not None:
        zeros = zeros.contiguous()
    if packed.numel():
        _done(lib().w4_pack(plan.handle, q.data_ptr(), scales.data_ptr(), _ptr(zeros),
                            packed.data_ptr(), stream), where)
    return W4Weight(packed, N, K, group, scales.dtype)


def linear_w4(x: torch.Tensor, weight: W4Weight, bias=None) -> torch.Tensor:
    """y = x @ W^T + bias for a packed 4-bit weight W [N, K] and x [..., K] of the
    type of its scales.  Sums are fp32 over the exact integers (sum x q less zero
    times sum x, so their error goes with |x| (q + zero)), scales applied per group
    in fp32, one rounding at the end.  Row i of y depends on row i
    of x and the weight alone, for every number of rows."""
    where = "linear_w4"
    dev = x.device
    if not (x.is_cuda and x.dtype == weight.dtype and x.dim() >= 1 and x.shape[-1] == weight.K
            and weight.packed.device == dev):
        raise ValueError(f"linear_w4: needs a {weight.dtype} CUDA tensor [..., {weight.K}] on "
                         f"{weight.packed.device}, got {tuple(x.shape)} {x.dtype} on {x.device}")
    N = weight.N
    bias = _bias32(where, bias, N, dev)
    _refuse_grad(where, x, bias)
    stream = _stream_of(where, dev)
    x = _dense(x)
    y = torch.empty(*x.shape[:-1], N, dtype=x.dtype, device=dev)
    M = x.numel() // weight.K
    if M:
        plan = _w4_plan(M, N, weight.K, x.dtype, weight.group)
        nws = plan.workspace_bytes
        ws = torch.empty(nws, dtype=torch.uint8, device=dev) if nws else None
        _done(lib().w4_run(plan.handle, x.data_ptr(), weight.packed.data_ptr(), _ptr(bias),
                           y.data_ptr(), _ptr(ws), nws, stream), where)
    return y


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
