"""Products grouped by expert, with group sizes that only the device knows.

    expert_order            a routing's slots sorted by expert: the groups
    fp8_grouped_gemm_b128   C[i] = A[tokens[i]] W_e^T for the rows i of expert e, E4M3 operands
    fp8_grouped_linear      a training step's expert layer on them, with its gradients

A prompt through a mixture of experts, with h the tokens' hidden states:

    o = expert_order(topk_ids, experts)
    q = fp8_quantize_b128(h)
    up = fp8_grouped_gemm_b128(q.codes, q.scales, w13.codes, w13.scales, o.offsets, tokens=o.tokens)
    ...
    down = fp8_grouped_gemm_b128(a.codes, a.scales, w2.codes, w2.scales, o.offsets, clear_rest=True)

and, for the weighted sum, row o.position[t, j] of ``down`` is token t's j-th expert's.  A slot of
no expert has a row behind the last group: ``clear_rest`` makes that a row of zeros (without it no
kernel writes it, and a weight of 0 does not remove a NaN that the memory held).
"""
from __future__ import annotations

import functools
from dataclasses import dataclass
from typing import Optional

import torch

from . import (_b128_operand, _borrow, _cdiv, _check, _dtype_code, _free_workspaces, _given, _matrix, _NoGradient, _raw_stream,
               B128_ROW, gemm_workspace, lib)


@dataclass
class ExpertOrder:
    offsets: torch.Tensor    # int32, experts + 1: expert e owns sorted rows offsets[e] .. offsets[e + 1] - 1
    order: torch.Tensor      # int32, slots: the slot of each sorted row
    tokens: torch.Tensor     # int32, slots: its token
    position: torch.Tensor   # int32, tokens x top_k: the sorted row of each slot


@functools.lru_cache(maxsize=4096)
def _order_workspace(tokens: int, top_k: int, experts: int) -> int:
    return lib().expert_order_workspace_bytes(tokens, top_k, experts)


def expert_order(topk_ids: torch.Tensor, experts: int, ws: Optional[torch.Tensor] = None) -> ExpertOrder:
    """The slots of a routing (topk_ids: int32 or int64, tokens x top_k) sorted by expert, in
    their order within one.  An id outside 0 .. experts - 1 names no expert: its slot comes
    behind all others', where no group is."""
    if experts >= 1 << 31 or topk_ids.dim() == 2 and topk_ids.shape[1] >= 1 << 31:
        raise ValueError("experts and the columns of topk_ids must be below 2^31")  # (the library takes them in 32 bits)
    ids = _matrix(topk_ids, "topk_ids")
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"topk_ids must be int32 or int64, not {ids.dtype}")
    tokens, top_k = ids.shape
    if top_k < 1:
        raise ValueError("topk_ids has no columns")
    new = ids.new_empty if ids.dtype == torch.int32 else lambda *s: ids.new_empty(s, dtype=torch.int32)
    n = tokens * top_k
    o = ExpertOrder(new(experts + 1 if experts > 0 else 0), new(n), new(n), new(tokens, top_k))
    stream, free = _raw_stream(ids.device), None
    if ws is not None:
        _given(ws, ids.device)
    elif n > 4096:
        ws, free = _borrow(_free_workspaces, gemm_workspace, ids.device, stream, _order_workspace(tokens, top_k, experts))
    rc = lib().expert_order(ids.data_ptr(), ids.dtype == torch.int64, tokens, top_k, experts, o.offsets.data_ptr(),
                            o.order.data_ptr(), o.tokens.data_ptr(), o.position.data_ptr(),
                            None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), stream)
    if rc:
        _check(rc)
    if free is not None:
        free.append(ws)
    return o


def _offsets(offsets: torch.Tensor, device) -> int:
    """Number of experts that `offsets` are of."""
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous() or offsets.device != device:
        raise ValueError("offsets must be contiguous int32 on the operands' device, one more than there are experts")
    return offsets.shape[0] - 1


def fp8_grouped_gemm_b128(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor, b_scales: torch.Tensor,
                          offsets: torch.Tensor, *, tokens: Optional[torch.Tensor] = None, out_dtype=torch.float32,
                          out: Optional[torch.Tensor] = None, clear_rest: bool = False) -> torch.Tensor:
    """C[i] = A_hat[tokens[i]] @ W_hat_e.T for offsets[e] <= i < offsets[e + 1].

    A: codes and row scales as fp8_quantize_b128 writes them.  W: codes experts x N x K with
    tile scales experts x ceil(N / 128) x ceil(K / 128), each expert's by itself; or both 2-D,
    the stacked matrix (experts * N) x K as ExpertWeights holds it.  ``tokens``: int32, one row
    of A per row of C (at most 2^28); without it row i of A is row i of C.  Rows that no group owns (expert_order
    puts slots of no expert there) get zeros with ``clear_rest``; without it they are left as they
    are in ``out``, and are uninitialized without one.  It has no gradient (fp8_grouped_linear has):
    a backward pass through scales that require one raises."""
    a_rows, k = _b128_operand(a_codes, a_scales, B128_ROW, "a")
    dev = a_codes.device
    experts = _offsets(offsets, dev)
    stacked = b_codes.dim() == 2
    if b_codes.dtype != torch.float8_e4m3fn or b_scales.dtype != torch.float32:
        raise TypeError("b: expected float8_e4m3fn codes and float32 scales")
    if b_codes.dim() != (2 if stacked else 3) or b_scales.dim() != b_codes.dim() or not b_codes.is_contiguous() or not b_scales.is_contiguous():
        raise ValueError("b_codes and b_scales must be contiguous, both 3-D (by expert) or both 2-D (stacked)")
    if experts < 1 or b_codes.shape[-1] != k or (b_codes.shape[0] % experts if stacked else b_codes.shape[0] != experts):
        raise ValueError(f"b_codes has shape {tuple(b_codes.shape)}; needed are {experts} experts and rows of {k}")
    n = b_codes.shape[0] // experts if stacked else b_codes.shape[1]
    want = (_cdiv(experts * n, 128), _cdiv(k, 128)) if stacked else (experts, _cdiv(n, 128), _cdiv(k, 128))
    if b_scales.shape != want:
        raise ValueError(f"b_scales has shape {tuple(b_scales.shape)}; codes {tuple(b_codes.shape)} need {want}")
    rows = a_rows
    if tokens is not None:
        if tokens.dtype != torch.int32 or tokens.dim() != 1 or not tokens.is_contiguous() or tokens.device != dev:
            raise ValueError("tokens must be contiguous 1-D int32 on the operands' device")
        rows = tokens.shape[0]
    if out is None:
        out = a_codes.new_empty((rows, n), dtype=out_dtype)
    elif out.shape != (rows, n) or not out.is_contiguous():
        raise ValueError(f"out must be contiguous, {rows} x {n}")
    if a_scales.device != dev or b_codes.device != dev or b_scales.device != dev or out.device != dev:
        raise ValueError("operands and out must be on one device")
    # An empty list of rows has no address: the call is none, but "without tokens" is another thing.
    call = lib().fp8_grouped_gemm_b128_cleared if clear_rest else lib().fp8_grouped_gemm_b128
    rc = call(a_codes.data_ptr(), a_scales.data_ptr(), a_rows, b_codes.data_ptr(), b_scales.data_ptr(), stacked,
              offsets.data_ptr(), experts, None if tokens is None else tokens.data_ptr() or offsets.data_ptr(), rows, n, k,
              out.data_ptr(), _dtype_code(out), _raw_stream(dev))
    if rc:
        _check(rc)
    if (a_scales.requires_grad or b_scales.requires_grad) and torch.is_grad_enabled():
        return _NoGradient.apply("fp8_grouped_gemm_b128", 1, out.detach(), a_scales, b_scales)
    return out


@functools.lru_cache(maxsize=4096)
def _sizes(rows, k, n, experts, want_dx, want_dw):
    """Bytes of (what the forward call saves, either call's workspace)."""
    l = lib()
    return (l.fp8_grouped_linear_saved_bytes(rows, k, n, experts, want_dx, want_dw),
            l.fp8_grouped_linear_workspace_bytes(rows, k, n, experts))


class _Fp8GroupedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, grad):
        # needs_input_grad goes by the inputs alone, whether a backward pass can follow or not.
        want_dx, want_dw = (need and grad for need in ctx.needs_input_grad[:2])
        dev = x.device
        experts, n, k = w.shape
        rows = x.shape[0]
        if not x.is_contiguous():
            x = x.contiguous()
        if not w.is_contiguous():
            w = w.contiguous()
        xt, wt = _dtype_code(x), _dtype_code(w)
        y = x.new_empty((rows, n))
        size, need = _sizes(rows, k, n, experts, want_dx, want_dw)
        saved = x.new_empty(size, dtype=torch.uint8) if size else None
        stream = _raw_stream(dev)
        ws, free = _borrow(_free_workspaces, gemm_workspace, dev, stream, max(need, 256))
        rc = lib().fp8_grouped_linear_forward(x.data_ptr(), xt, w.data_ptr(), wt, offsets.data_ptr(), experts, rows, k, n,
                                              y.data_ptr(), want_dx, want_dw, None if saved is None else saved.data_ptr(),
                                              size, ws.data_ptr(), ws.numel(), stream)
        if rc:
            _check(rc)
        if free is not None:
            free.append(ws)
        if want_dx or want_dw:
            ctx.save_for_backward(saved, offsets)
            ctx.sizes = rows, k, n, experts, xt, wt, w.dtype, need
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        want_dx, want_dw = ctx.needs_input_grad[:2]
        rows, k, n, experts, xt, wt, w_dtype, need = ctx.sizes
        saved, offsets = ctx.saved_tensors
        dev = dy.device
        if not dy.is_contiguous():
            dy = dy.contiguous()
        dx = dy.new_empty((rows, k)) if want_dx else None
        dw = dy.new_empty((experts, n, k), dtype=w_dtype) if want_dw else None
        stream = _raw_stream(dev)
        ws, free = _borrow(_free_workspaces, gemm_workspace, dev, stream, max(need, 256))
        # An empty gradient has no address of its own: any aligned one stands for it.
        rc = lib().fp8_grouped_linear_backward(dy.data_ptr(), xt, wt, offsets.data_ptr(), experts, rows, k, n,
                                               (dx.data_ptr() or ws.data_ptr()) if want_dx else None,
                                               (dw.data_ptr() or ws.data_ptr()) if want_dw else None,
                                               None if saved is None else saved.data_ptr(),
                                               0 if saved is None else saved.numel(), ws.data_ptr(), ws.numel(), stream)
        if rc:
            _check(rc)
        if free is not None:
            free.append(ws)
        return dx, dw, None, None


def fp8_grouped_linear(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor) -> torch.Tensor:
    """x (rows x in-features, the rows by expert) times each expert's matrix of w (experts x
    out-features x in-features) transposed, both bfloat16 or float32, on 8-bit block-128
    operands; differentiable in both.  Expert e owns rows offsets[e] .. offsets[e + 1] - 1
    (int32, as expert_order gives them, or a run of those for a run of the experts; read on the
    device); rows before the first group and behind the last are zeros in y and dx.  y and dx
    have x's dtype, dw has w's.  ``offsets`` must not be written before the backward pass."""
    if x.dim() != 2 or w.dim() != 3 or x.shape[1] != w.shape[2]:
        raise ValueError(f"x has shape {tuple(x.shape)}, w {tuple(w.shape)}: needed are rows x in and experts x out x in")
    if x.device != w.device or not x.is_cuda:
        raise ValueError("x and w must be on one device")
    if _offsets(offsets, x.device) != w.shape[0] or w.shape[0] < 1:
        raise ValueError(f"offsets are of {offsets.shape[0] - 1} experts, w has {w.shape[0]}")
    return _Fp8GroupedLinear.apply(x, w, offsets, torch.is_grad_enabled())
