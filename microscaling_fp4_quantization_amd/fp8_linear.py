"""A linear layer on 8-bit block-128 operands, with its gradients.

    y  = Qr(x) Qt(w)^T
    dx = Qr(dy) Qt(w)
    dw = Qr(dy^T) Qr(x^T)^T

Qr and Qt are the values that fp8_quantize_b128 gives under row and tile scales.
The quantizer is taken as the identity in the backward pass (its slope inside the
range is 1 on average): dx and dw are the exact gradients of the product, with each
product's operands quantized along its own contraction.  Each tensor is read once:
x and dy give the row-major and the transposed codes in one pass, and w's tile
scales serve both products that it is in.  Each pass is one call of the library: a
training step's small layers are bound by the host, and call by call the same work
took it half as long again.
"""
from __future__ import annotations

import functools
import math

import torch

from . import _borrow, _check, _dtype_code, _free_workspaces, _raw_stream, gemm_workspace, lib


@functools.lru_cache(maxsize=4096)
def _sizes(tokens, k, out, xt, wt, want_dx, want_dw):
    """Bytes of (what the forward call saves, either call's workspace)."""
    l = lib()
    return (l.fp8_linear_saved_bytes(tokens, k, out, want_dx, want_dw),
            l.fp8_linear_workspace_bytes(tokens, k, out, xt, wt))


class _Fp8Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, grad):
        # needs_input_grad goes by the inputs alone, whether a backward pass can follow or not.
        want_dx, want_dw = (need and grad for need in ctx.needs_input_grad[:2])
        dev = x.device
        out, k = w.shape
        shape = x.shape
        if x.dim() != 2:
            x = x.reshape(math.prod(shape[:-1]), k)
        if not x.is_contiguous():
            x = x.contiguous()
        if not w.is_contiguous():
            w = w.contiguous()
        tokens = x.shape[0]
        xt, wt = _dtype_code(x), _dtype_code(w)
        y = x.new_empty((tokens, out))
        n, need = _sizes(tokens, k, out, xt, wt, want_dx, want_dw)
        saved = x.new_empty(n, dtype=torch.uint8) if n else None
        stream = _raw_stream(dev)
        ws, free = _borrow(_free_workspaces, gemm_workspace, dev, stream, need)
        rc = lib().fp8_linear_forward(x.data_ptr(), xt, w.data_ptr(), wt, tokens, k, out, y.data_ptr(), want_dx, want_dw,
                                      None if saved is None else saved.data_ptr(), n, ws.data_ptr(), ws.numel(), stream)
        if rc:
            _check(rc)
        if free is not None:
            free.append(ws)
        if want_dx or want_dw:
            ctx.save_for_backward(saved)
            ctx.sizes = shape, tokens, k, out, xt, wt, w.dtype, need
        return y if len(shape) == 2 else y.view(*shape[:-1], out)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        want_dx, want_dw = ctx.needs_input_grad[:2]
        shape, tokens, k, out, xt, wt, w_dtype, need = ctx.sizes
        saved, = ctx.saved_tensors
        dev = dy.device
        if not dy.is_contiguous():
            dy = dy.contiguous()
        dx = dy.new_empty(shape) if want_dx else None
        dw = dy.new_empty((out, k), dtype=w_dtype) if want_dw else None
        stream = _raw_stream(dev)
        ws, free = _borrow(_free_workspaces, gemm_workspace, dev, stream, need)
        # An empty gradient has no address of its own: any aligned one stands for it.
        rc = lib().fp8_linear_backward(dy.data_ptr(), xt, wt, tokens, k, out,
                                       (dx.data_ptr() or ws.data_ptr()) if want_dx else None,
                                       (dw.data_ptr() or ws.data_ptr()) if want_dw else None,
                                       None if saved is None else saved.data_ptr(), 0 if saved is None else saved.numel(),
                                       ws.data_ptr(), ws.numel(), stream)
        if rc:
            _check(rc)
        if free is not None:
            free.append(ws)
        return dx, dw, None


def fp8_linear(x: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
    """x (... x in-features) times w (out-features x in-features) transposed, both
    bfloat16 or float32 on the device, on 8-bit block-128 operands; differentiable in
    both.  y and dx have x's dtype, dw has w's."""
    if w.dim() != 2 or x.dim() < 1 or x.shape[-1] != w.shape[1]:
        raise ValueError(f"x has shape {tuple(x.shape)}, w {tuple(w.shape)}: the last sizes must agree")
    if x.device != w.device or not x.is_cuda:
        raise ValueError("x and w must be on one device")
    return _Fp8Linear.apply(x, w, torch.is_grad_enabled())
