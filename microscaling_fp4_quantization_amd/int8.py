"""8-bit integer operands with one scale per row, their product and a served linear layer.

    s = max(RN32(max |x| / 127), 2^-126) of a row,  code = RN32(x / s) to the nearest whole number
    C[m][n] = acc sa[m] sb[n] + bias[n],  acc = sum over k of A[m][k] B[n][k], exact

Activations have a scale per token, weights one per output channel.  An element of C is
a function of its own row, column, scales and bias: its bits do not change with the
batch that a token is in.
"""
from __future__ import annotations

import functools
import math
from dataclasses import dataclass
from typing import Optional

import torch

from . import _borrow, _cdiv, _check, _dtype_code, _free_workspaces, _given, _matrix, _NoGradient, _raw_stream, gemm_workspace, lib


@dataclass
class Int8Quantized:
    codes: torch.Tensor    # int8, rows x cols rounded up to 16
    scales: torch.Tensor   # float32, one per row


def int8_quantize_rows(x: torch.Tensor, *, out: Optional[Int8Quantized] = None) -> Int8Quantized:
    """int8 codes of x (rows x cols, bfloat16 or float32) with one float32 scale per row.
    ``out``: preallocated outputs, laid out as the call returns them."""
    x = _matrix(x)
    rows, cols = x.shape
    shape = rows, _cdiv(cols, 16) * 16
    if out is None:
        out = Int8Quantized(x.new_empty(shape, dtype=torch.int8), x.new_empty(rows, dtype=torch.float32))
    else:
        for t, want, dt, name in ((out.codes, shape, torch.int8, "codes"), (out.scales, (rows,), torch.float32, "scales")):
            if t.shape != want or t.dtype != dt or t.device != x.device or not t.is_contiguous():
                raise ValueError(f"out.{name} must be a contiguous {dt} tensor of shape {want} on {x.device}")
    rc = lib().int8_quantize_rows(x.data_ptr(), _dtype_code(x), rows, cols, out.codes.data_ptr(), out.scales.data_ptr(),
                                  _raw_stream(x.device))
    if rc:
        _check(rc)
    return out


def _operand(codes: torch.Tensor, scales: torch.Tensor, what: str):
    _matrix(codes, what + "_codes")
    if codes.dtype != torch.int8 or scales.dtype != torch.float32:
        raise TypeError(f"{what}: expected int8 codes and float32 scales")
    if scales.shape != codes.shape[:1] or not scales.is_contiguous():
        raise ValueError(f"{what}_scales must be contiguous, one per row of {what}_codes ({codes.shape[0]})")
    return codes.shape


def _bias(bias: Optional[torch.Tensor], n: int, dev):
    """(address, dtype code) of a bias."""
    if bias is None:
        return None, 0
    if bias.shape != (n,) or not bias.is_contiguous() or bias.device != dev:
        raise ValueError(f"bias must be contiguous, {n} elements, on the codes' device")
    return bias.data_ptr(), _dtype_code(bias)


def _result(name: str, out: torch.Tensor, *inputs):
    """out, refusing a backward pass where an input requires a gradient."""
    if torch.is_grad_enabled():
        wanted = [t for t in inputs if t is not None and t.requires_grad]
        if wanted:
            return _NoGradient.apply(name, 1, out.detach(), *wanted)
    return out


def int8_gemm(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor, b_scales: torch.Tensor,
              bias: Optional[torch.Tensor] = None, out_dtype=torch.float32, out: Optional[torch.Tensor] = None,
              ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C = A_hat @ B_hat.T + bias for operands as int8_quantize_rows writes them.  It has no
    gradient: a backward pass through scales or a bias that require one raises."""
    m, k = _operand(a_codes, a_scales, "a")
    n, kb = _operand(b_codes, b_scales, "b")
    if kb != k:
        raise ValueError(f"a_codes has rows of {k}, b_codes of {kb}")
    dev = a_codes.device
    if out is None:
        out = a_codes.new_empty((m, n), dtype=out_dtype)
    elif out.shape != (m, n) or not out.is_contiguous():
        raise ValueError(f"out must be contiguous, {m} x {n}")
    if a_scales.device != dev or b_codes.device != dev or b_scales.device != dev or out.device != dev:
        raise ValueError("operands and out must be on one device")
    bp, bt = _bias(bias, n, dev)
    l, ct = lib(), _dtype_code(out)
    stream, free = _raw_stream(dev), None
    if ws is not None:
        _given(ws, dev)
    elif m > 16:  # at most 16 rows take none
        need = l.int8_gemm_workspace_bytes(m, n, k)
        if need:
            ws, free = _borrow(_free_workspaces, gemm_workspace, dev, stream, need)
    rc = l.int8_gemm(a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(), b_scales.data_ptr(), bp, bt, m, n, k,
                     out.data_ptr(), ct, None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), stream)
    if rc:
        _check(rc)
    if free is not None:
        free.append(ws)
    return _result("int8_gemm", out, a_scales, b_scales, bias)


@functools.lru_cache(maxsize=4096)
def _linear_workspace(tokens: int, k: int, n: int) -> int:
    return lib().int8_linear_workspace_bytes(tokens, k, n)


def int8_linear(x: torch.Tensor, w: Int8Quantized, bias: Optional[torch.Tensor] = None, out_dtype=None,
                out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x (... x in-features, bfloat16 or float32), quantized per token, times w (out-features x
    in-features as int8_quantize_rows writes it) transposed, plus bias; in x's dtype unless
    ``out_dtype`` or ``out`` (tokens x out-features) says otherwise.  For serving: a backward
    pass through it raises."""
    n, kp = _operand(w.codes, w.scales, "w")
    shape = x.shape
    if len(shape) < 1 or _cdiv(shape[-1], 16) * 16 != kp:
        raise ValueError(f"x has shape {tuple(shape)}, w's rows {kp} codes: in-features rounded up to 16 must agree")
    k = shape[-1]
    dev = x.device
    if not x.is_cuda or w.codes.device != dev or w.scales.device != dev:
        raise ValueError("x and w must be on one device")
    m = shape[0] if len(shape) == 2 else math.prod(shape[:-1])
    xc = x if x.is_contiguous() else x.contiguous()
    given = out is not None
    if not given:
        out = x.new_empty((m, n), dtype=out_dtype or x.dtype)
    elif out.shape != (m, n) or not out.is_contiguous() or out.device != dev:
        raise ValueError(f"out must be contiguous, {m} x {n}, on x's device")
    bp, bt = _bias(bias, n, dev)
    stream, free = _raw_stream(dev), None
    if ws is not None:
        _given(ws, dev)
    else:
        need = _linear_workspace(m, k, n)
        if need:
            ws, free = _borrow(_free_workspaces, gemm_workspace, dev, stream, need)
    rc = lib().int8_linear(xc.data_ptr(), _dtype_code(xc), w.codes.data_ptr(), w.scales.data_ptr(), bp, bt, m, k, n,
                           out.data_ptr(), _dtype_code(out), None if ws is None else ws.data_ptr(),
                           0 if ws is None else ws.numel(), stream)
    if rc:
        _check(rc)
    if free is not None:
        free.append(ws)
    y = _result("int8_linear", out, x, w.scales, bias)
    return y if given or len(shape) == 2 else y.view(*shape[:-1], n)
