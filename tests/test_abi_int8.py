"""The 8-bit integer entry points refuse bad arguments before any launch (no GPU is
touched: every call fails validation or is an empty no-op)."""
import pytest
import torch

import microscaling_fp4_quantization_amd as fq
from test_abi import L, err  # noqa: F401  (the loaded library, built if it is missing)

OK, ARG, SHAPE, ALIGN, WS = 0, 1, 2, 3, 4
A, B, C, D = 0x10000, 0x20000, 0x30000, 0x40000  # aligned addresses, never dereferenced


def test_quantize_validation(L):
    def q(x=A, xt=0, rows=4, cols=40, codes=B, scales=C):
        return L.int8_quantize_rows(x, xt, rows, cols, codes, scales, None)

    assert q(xt=2) == ARG and "dtype" in err(L)
    assert q(rows=-1) == SHAPE and q(cols=-1) == SHAPE
    assert q(rows=1 << 31, cols=1) == SHAPE and q(rows=1 << 30, cols=1 << 30) == SHAPE and "limit" in err(L)
    assert q(x=None) == ARG and q(codes=None) == ARG and q(scales=None) == ARG
    assert q(x=A + 1) == ALIGN and q(xt=1, x=A + 2) == ALIGN and q(codes=B + 8) == ALIGN and q(scales=C + 2) == ALIGN
    assert q(rows=0, x=None, codes=None, scales=None) == OK


def test_gemm_validation(L):
    def gemm(a=A, sa=B, b=C, sb=D, bias=None, bt=0, m=4, n=8, k=64, c=A, ct=0, ws=None, wsb=0):
        return L.int8_gemm(a, sa, b, sb, bias, bt, m, n, k, c, ct, ws, wsb, None)

    assert gemm(ct=2) == ARG and gemm(bias=A, bt=3) == ARG
    assert gemm(m=-1) == SHAPE and gemm(n=1 << 21) == SHAPE and gemm(m=1 << 31) == SHAPE
    assert gemm(k=24) == SHAPE and "multiple of 16" in err(L)
    assert gemm(k=1 << 17) == SHAPE and "2^31" in err(L)
    for missing in ("a", "sa", "b", "sb", "c"):
        assert gemm(**{missing: None}) == ARG, missing
    assert gemm(a=A + 8) == ALIGN and gemm(b=C + 4) == ALIGN and gemm(sa=B + 2) == ALIGN and gemm(c=A + 1) == ALIGN
    assert gemm(bias=A + 2, bt=1) == ALIGN and gemm(ct=1, c=A + 2) == ALIGN
    assert gemm(m=0, a=None, sa=None, b=None, sb=None, c=None) == OK
    assert gemm(n=0, a=None, sa=None, b=None, sb=None, c=None) == OK
    need = L.int8_gemm_workspace_bytes(100, 256, 8192)
    assert need > 0 and need % (4 * 100 * 256) == 0
    assert gemm(m=100, n=256, k=8192) == WS and gemm(m=100, n=256, k=8192, ws=A, wsb=need - 1) == WS
    assert gemm(m=100, n=256, k=8192, ws=A + 8, wsb=need) == ALIGN
    assert L.int8_gemm_workspace_bytes(16, 256, 8192) == 0 and L.int8_gemm_workspace_bytes(0, 256, 8192) == 0
    assert L.int8_gemm_workspace_bytes(100, 256, 8200) == 0


def test_linear_validation(L):
    need = L.int8_linear_workspace_bytes(40, 100, 70)
    assert need >= 40 * 112 + 160
    assert L.int8_linear_workspace_bytes(1, 18944, 70) == 0 and L.int8_linear_workspace_bytes(2, 18944, 70) >= 2 * 18944

    def lin(x=A, xt=0, w=B, sw=C, bias=None, bt=0, t=40, k=100, n=70, y=D, yt=0, ws=A, wsb=need):
        return L.int8_linear(x, xt, w, sw, bias, bt, t, k, n, y, yt, ws, wsb, None)

    assert lin(xt=2) == ARG and lin(yt=2) == ARG and lin(bias=A, bt=2) == ARG
    assert lin(t=-1) == SHAPE and lin(k=131057) == SHAPE and lin(k=-1) == SHAPE and lin(n=1 << 21) == SHAPE
    assert lin(k=1 << 62) == SHAPE
    for missing in ("x", "w", "sw", "y"):
        assert lin(**{missing: None}) == ARG, missing
    assert lin(x=A + 1) == ALIGN and lin(w=B + 8) == ALIGN and lin(sw=C + 2) == ALIGN and lin(yt=1, y=D + 2) == ALIGN
    assert lin(ws=None) == WS and lin(wsb=need - 1) == WS and lin(ws=A + 16) == ALIGN
    assert lin(t=0, x=None, w=None, sw=None, y=None, ws=None, wsb=0) == OK
    assert L.int8_linear_workspace_bytes(0, 100, 70) == 0 and L.int8_linear_workspace_bytes(4, 131057, 70) == 0


def test_binding_refuses():
    i8, f32 = (lambda *s: torch.zeros(s, dtype=torch.int8)), (lambda *s: torch.zeros(s))
    with pytest.raises(ValueError, match="device"):
        fq.int8_quantize_rows(f32(4, 8))
    with pytest.raises(ValueError, match="2-D"):
        fq.int8_quantize_rows(f32(8))
    with pytest.raises(ValueError, match="device"):
        fq.int8_gemm(i8(4, 16), f32(4), i8(8, 16), f32(8))
    with pytest.raises(ValueError, match="device"):
        fq.int8_linear(f32(4, 16), fq.Int8Quantized(i8(8, 16), f32(8)))
