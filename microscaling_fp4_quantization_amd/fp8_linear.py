"""A linear layer on 8-bit block-128 operands, with its gradients.

    y  = Qr(x) Qt(w)^T
    dx = Qr(dy) Qt(w)
    dw = Qr(dy^T) Qr(x^T)^T

Qr and Qt are the values that fp8_quantize_b128 gives under row and tile scales.
The quantizer is taken as the identity in the backward pass (its slope inside the
range is 1 on average): dx and dw are the exact gradients of the product, with each
product's operands quantized along its own contraction.  Each tensor is read once:
x and dy give the row-major and the transposed codes in one pass, and w's tile
scales serve both products that it is in.
"""
from __future__ import annotations

import torch

from . import B128_ROW, B128_TILE, fp8_gemm_b128, fp8_quantize_b128


class _Fp8Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w):
        need_dx, need_dw = ctx.needs_input_grad
        flat = x.reshape(-1, x.shape[-1]).contiguous()
        xq = fp8_quantize_b128(flat, B128_ROW, transposed=need_dw)
        wq = fp8_quantize_b128(w.contiguous(), B128_TILE, transposed=need_dx)
        if need_dx or need_dw:
            ctx.save_for_backward(wq.codes_t, wq.scales_t, xq.codes_t, xq.scales_t)
            ctx.x_shape, ctx.x_dtype, ctx.w_dtype = x.shape, x.dtype, w.dtype
        y = fp8_gemm_b128(xq.codes, xq.scales, wq.codes, wq.scales, B128_TILE, out_dtype=x.dtype)
        return y if x.dim() == 2 else y.view(*x.shape[:-1], w.shape[0])

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        need_dx, need_dw = ctx.needs_input_grad
        wt, swt, xt, sxt = ctx.saved_tensors
        dy = dy.reshape(-1, dy.shape[-1]).contiguous()
        q = fp8_quantize_b128(dy, B128_ROW, codes=need_dx, transposed=need_dw)
        dx = dw = None
        if need_dx:
            dx = fp8_gemm_b128(q.codes, q.scales, wt, swt, B128_TILE, out_dtype=ctx.x_dtype).view(ctx.x_shape)
        if need_dw:
            dw = fp8_gemm_b128(q.codes_t, q.scales_t, xt, sxt, B128_ROW, out_dtype=ctx.w_dtype)
        return dx, dw


def fp8_linear(x: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
    """x (... x in-features) times w (out-features x in-features) transposed, both
    bfloat16 or float32, on 8-bit block-128 operands; differentiable in both.  y
    and dx have x's dtype, dw has w's."""
    if w.dim() != 2 or x.dim() < 1 or x.shape[-1] != w.shape[1]:
        raise ValueError(f"x has shape {tuple(x.shape)}, w {tuple(w.shape)}: the last sizes must agree")
    if x.device != w.device:
        raise ValueError("x and w must be on one device")
    return _Fp8Linear.apply(x, w)
