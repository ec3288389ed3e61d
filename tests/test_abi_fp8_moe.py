"""The 8-bit block-128 and mixture-of-experts entry points refuse bad arguments
before any launch (no GPU is touched: every call fails validation or is an empty
no-op)."""
import ctypes

import pytest

import microscaling_fp4_quantization_amd as fq
from test_abi import L, err  # noqa: F401  (the loaded library, built if it is missing)

OK, ARG, SHAPE, ALIGN, WS = 0, 1, 2, 3, 4
A, B, C, D = 0x10000, 0x20000, 0x30000, 0x40000  # aligned addresses, never dereferenced


def quant(L, x=A, xt=0, rows=4, cols=64, kind=0, codes=B, scales=C, codes_t=None, scales_t=None):
    return L.fp8_quantize_b128(x, xt, rows, cols, kind, codes, scales, codes_t, scales_t, None)


def test_quantize_validation(L):
    assert quant(L, xt=2) == ARG and "dtype" in err(L)
    assert quant(L, kind=2) == ARG and "kind" in err(L)
    assert quant(L, rows=-1) == SHAPE
    assert quant(L, rows=1 << 40, cols=1 << 22) == SHAPE and "limit" in err(L)
    assert quant(L, x=None) == ARG
    assert quant(L, codes=None, scales=None) == ARG and "both" in err(L)
    assert quant(L, scales=None) == ARG
    assert quant(L, codes_t=D) == ARG and "scales_t" in err(L)
    assert quant(L, x=A + 1) == ALIGN
    assert quant(L, xt=1, x=A + 2) == ALIGN
    assert quant(L, codes=B + 8) == ALIGN
    assert quant(L, scales=C + 2) == ALIGN
    assert quant(L, codes_t=D + 4, scales_t=D) == ALIGN
    assert quant(L, rows=0, x=None, codes=None, scales=None) == OK
    assert quant(L, cols=0, x=None, codes=None, scales=None) == OK


def gemm(L, a=A, sa=B, b=C, sb=D, kind=1, m=4, n=8, k=64, c=A, ct=0, ws=None, wsb=0):
    return L.fp8_gemm_b128(a, sa, b, sb, kind, m, n, k, c, ct, ws, wsb, None)


def test_gemm_validation(L):
    assert gemm(L, kind=-1) == ARG and "kind" in err(L)
    assert gemm(L, ct=3) == ARG
    assert gemm(L, m=-1) == SHAPE
    assert gemm(L, k=24) == SHAPE and "multiple of 16" in err(L)
    assert gemm(L, k=(1 << 22) + 16) == SHAPE
    assert gemm(L, n=1 << 22) == SHAPE
    assert gemm(L, n=1 << 21, ct=1) == SHAPE
    assert gemm(L, m=1 << 31) == SHAPE
    for missing in ("a", "sa", "b", "sb", "c"):
        assert gemm(L, **{missing: None}) == ARG, missing
    assert gemm(L, a=A + 8) == ALIGN and gemm(L, b=C + 4) == ALIGN
    assert gemm(L, sa=B + 2) == ALIGN and gemm(L, c=A + 1) == ALIGN
    assert gemm(L, m=0, a=None, sa=None, b=None, sb=None, c=None) == OK
    assert gemm(L, n=0, a=None, sa=None, b=None, sb=None, c=None) == OK
    need = L.fp8_gemm_b128_workspace_bytes(100, 256, 8192, 0)
    assert need > 0 and need % (4 * 100 * 256) == 0
    assert gemm(L, m=100, n=256, k=8192) == WS
    assert gemm(L, m=100, n=256, k=8192, ws=A, wsb=need - 1) == WS
    assert gemm(L, m=100, n=256, k=8192, ws=A + 8, wsb=need) == ALIGN
    assert L.fp8_gemm_b128_workspace_bytes(16, 256, 8192, 0) == 0
    assert L.fp8_gemm_b128_workspace_bytes(0, 256, 8192, 0) == 0


def weights(codes=A, scales=B, g=None, n=0):
    return fq._ExpertWeightsC(codes, scales, g, n)


def moe(L, x=A, xt=0, t=4, d=64, i=32, e=6, k=2, fmt=0, w13=None, w2=None, router=B, rt=0, ids=C, wts=D, y=A, yt=0,
        ws=A, wsb=1 << 30):
    ref = lambda w: None if w is None else ctypes.byref(w)
    return L.moe_layer(x, xt, t, d, i, e, k, fmt, ref(w13 or weights()), ref(w2 or weights()), router, rt, 1, ids, wts,
                       y, yt, ws, wsb, None)


def test_moe_validation(L):
    assert moe(L, xt=2) == ARG and moe(L, yt=2) == ARG and moe(L, rt=2) == ARG
    assert moe(L, fmt=2) == ARG and "fmt" in err(L)
    assert moe(L, t=65) == SHAPE and "tokens" in err(L)
    assert moe(L, t=-1) == SHAPE
    assert moe(L, d=48) == SHAPE and moe(L, i=16) == SHAPE and moe(L, d=0) == SHAPE and moe(L, i=(1 << 20) + 32) == SHAPE
    assert moe(L, e=513) == SHAPE and moe(L, e=0) == SHAPE
    assert moe(L, k=7) == SHAPE and moe(L, k=0) == SHAPE and moe(L, e=40, k=17) == SHAPE
    assert moe(L, w13=weights(codes=None)) == ARG and moe(L, w2=weights(scales=None)) == ARG
    assert moe(L, w13=weights(codes=A + 8)) == ALIGN
    assert moe(L, fmt=1, w2=weights(scales=B + 1)) == ALIGN and moe(L, fmt=3, w2=weights(scales=B + 2)) == ALIGN
    assert moe(L, w13=weights(g=C, n=1)) == ARG and "UE4M3 only" in err(L)
    assert moe(L, fmt=1, w13=weights(g=C, n=3)) == ARG and "one per expert" in err(L)
    assert moe(L, fmt=1, w13=weights(g=C + 2, n=6)) == ALIGN
    for missing in ("x", "ids", "wts", "y"):
        assert moe(L, **{missing: None}) == ARG, missing
    assert moe(L, x=A + 8) == ALIGN and moe(L, router=B + 4) == ALIGN and moe(L, yt=1, y=A + 2) == ALIGN
    need = L.moe_layer_workspace_bytes(4, 64, 32, 6, 2)
    assert need > 0
    assert moe(L, ws=None) == WS and moe(L, wsb=need - 1) == WS and moe(L, ws=A + 16) == ALIGN
    assert L.moe_layer_workspace_bytes(0, 64, 32, 6, 2) == 0 and L.moe_layer_workspace_bytes(65, 64, 32, 6, 2) == 0
    assert L.moe_layer(None, 0, 0, 64, 32, 6, 2, 0, None, None, None, 0, 1, None, None, None, 0, None, 0, None) == OK
    assert L.moe_layer(A, 0, 4, 64, 32, 6, 2, 0, None, None, None, 0, 1, C, D, A, 0, A, need, None) == ARG
    assert moe(L, fmt=1, w13=weights(scales=B, g=C, n=1), ws=None) == WS  # past the weights' checks


def test_linear_validation(L):
    T, K, N = 40, 96, 70
    saved, ws = L.fp8_linear_saved_bytes(T, K, N, 1, 1), L.fp8_linear_workspace_bytes(T, K, N, 0, 0)
    assert saved > 0 and ws > 0 and saved % 256 == 0
    assert L.fp8_linear_saved_bytes(T, K, N, 0, 0) == 0 and L.fp8_linear_saved_bytes(-1, K, N, 1, 1) == 0
    assert L.fp8_linear_saved_bytes(T, K, N, 1, 0) + L.fp8_linear_saved_bytes(T, K, N, 0, 1) == saved

    def fwd(x=A, xt=0, w=B, wt=0, t=T, k=K, n=N, y=C, dx=1, dw=1, s=D, sb=saved, wk=A, wb=ws):
        return L.fp8_linear_forward(x, xt, w, wt, t, k, n, y, dx, dw, s, sb, wk, wb, None)

    assert fwd(xt=2) == ARG and fwd(wt=-1) == ARG
    assert fwd(t=-1) == SHAPE and fwd(n=1 << 21) == SHAPE and fwd(t=1 << 20, k=1 << 20) == SHAPE
    assert fwd(x=None) == ARG and fwd(w=None) == ARG and fwd(y=None) == ARG
    assert fwd(x=A + 1) == ALIGN and fwd(y=C + 1) == ALIGN and fwd(wt=1, w=B + 2) == ALIGN
    assert fwd(s=None) == WS and fwd(sb=saved - 1) == WS and "saved" in err(L)
    assert fwd(s=D + 16) == ALIGN
    assert fwd(wk=None) == WS and fwd(wb=100) == WS and fwd(wk=A + 16) == ALIGN

    def bwd(dy=A, xt=0, wt=0, t=T, k=K, n=N, dx=B, dw=C, s=D, sb=saved, wk=A, wb=ws):
        return L.fp8_linear_backward(dy, xt, wt, t, k, n, dx, dw, s, sb, wk, wb, None)

    assert bwd(dx=None, dw=None) == ARG and "both" in err(L)
    assert bwd(dy=None) == ARG and bwd(xt=3) == ARG and bwd(k=-1) == SHAPE
    assert bwd(dx=B + 1) == ALIGN and bwd(wt=1, dw=C + 2) == ALIGN
    assert bwd(s=None) == WS and bwd(sb=saved - 1) == WS and bwd(wk=None) == WS and bwd(wb=1) == WS
