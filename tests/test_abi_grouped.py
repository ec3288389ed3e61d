"""The grouped entry points refuse bad arguments before any launch (no GPU is touched:
every call fails validation or is an empty no-op)."""
import pytest
import torch

import microscaling_fp4_quantization_amd as fq
from test_abi import L, err  # noqa: F401  (the loaded library, built if it is missing)

OK, ARG, SHAPE, ALIGN, WS = 0, 1, 2, 3, 4
A, B, C, D, E, F = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000  # aligned addresses, never dereferenced


def test_order_validation(L):
    def order(ids=A, wide=0, t=4, k=2, e=8, off=B, o=C, tok=D, pos=E, ws=None, wsb=0):
        return L.expert_order(ids, wide, t, k, e, off, o, tok, pos, ws, wsb, None)

    assert order(e=0) == SHAPE and order(e=513) == SHAPE and "experts" in err(L)
    assert order(t=-1) == SHAPE and order(k=0) == SHAPE and order(t=1 << 30, k=2) == SHAPE
    for missing in ("ids", "off", "o", "tok", "pos"):
        assert order(**{missing: None}) == ARG, missing
    assert order(ids=A + 2) == ALIGN and order(ids=A + 4, wide=1) == ALIGN and order(pos=E + 1) == ALIGN
    assert L.expert_order_workspace_bytes(2048, 2, 8) == 0 and L.expert_order_workspace_bytes(-1, 2, 8) == 0
    need = L.expert_order_workspace_bytes(16384, 8, 128)
    assert need > 0 and need % (4 * 129) == 0
    assert order(t=16384, k=8, e=128) == WS and order(t=16384, k=8, e=128, ws=A, wsb=need - 1) == WS
    assert order(t=16384, k=8, e=128, ws=A + 2, wsb=need) == ALIGN


def test_gemm_validation(L):
    def gemm(a=A, sa=B, ar=40, b=C, sb=D, st=0, off=E, e=4, tok=None, r=40, n=96, k=64, c=F, ct=0):
        return L.fp8_grouped_gemm_b128(a, sa, ar, b, sb, st, off, e, tok, r, n, k, c, ct, None)

    assert gemm(ct=2) == ARG and gemm(e=0) == SHAPE and gemm(e=513) == SHAPE
    assert gemm(r=-1, ar=-1) == SHAPE and gemm(k=24) == SHAPE and gemm(k=(1 << 22) + 16) == SHAPE
    assert gemm(n=1 << 22) == SHAPE and gemm(n=1 << 21, ct=1) == SHAPE and gemm(r=1 << 31, ar=1 << 31) == SHAPE
    assert gemm(ar=39) == SHAPE and "agree" in err(L)
    assert gemm(tok=A, ar=1 << 26, k=32) == SHAPE and "2^31" in err(L)
    assert gemm(tok=A, ar=1 << 29, k=0) == SHAPE
    for missing in ("a", "sa", "b", "sb", "off", "c"):
        assert gemm(**{missing: None}) == ARG, missing
    assert gemm(a=A + 8) == ALIGN and gemm(b=C + 4) == ALIGN and gemm(sb=D + 2) == ALIGN and gemm(c=F + 1) == ALIGN
    assert gemm(off=E + 2) == ALIGN and gemm(tok=A + 2) == ALIGN
    assert gemm(r=0, ar=0, a=None, sa=None, b=None, sb=None, off=None, c=None) == OK
    assert gemm(n=0, a=None, sa=None, b=None, sb=None, off=None, c=None) == OK


@pytest.mark.parametrize("tokens", [None, A])
def test_gemm_rows_that_the_groups_tiles_cannot_count(L, tokens):
    """512 groups that all hold every row (offsets out of order) take 2^22 tiles of 64 rows each at
    2^28 rows: 2^30 for 256 of them, a sum that 32 bits hold; more rows are refused."""
    for rows in ((1 << 28) + 1, 1 << 30, (1 << 31) - 1):
        got = L.fp8_grouped_gemm_b128(A, B, 1 if tokens else rows, C, D, 0, E, 4, tokens, rows, 1, 16, F, 0, None)
        assert got == SHAPE and "2^28" in err(L), rows


def test_linear_validation(L):
    T, K, N, X = 40, 96, 70, 3
    saved, ws = L.fp8_grouped_linear_saved_bytes(T, K, N, X, 1, 1), L.fp8_grouped_linear_workspace_bytes(T, K, N, X)
    assert saved > 0 and ws > 0 and saved % 256 == 0
    assert L.fp8_grouped_linear_saved_bytes(T, K, N, X, 0, 0) == 0 and L.fp8_grouped_linear_saved_bytes(-1, K, N, X, 1, 1) == 0
    assert L.fp8_grouped_linear_saved_bytes(T, K, N, X, 1, 0) + L.fp8_grouped_linear_saved_bytes(T, K, N, X, 0, 1) == saved
    # x's transpose: at most (40 + 3 * 127) / 128 = 3 blocks of the groups
    assert L.fp8_grouped_linear_saved_bytes(T, K, N, X, 0, 1) == K * 3 * 128 + (4 * K * 3 + 255) // 256 * 256

    def fwd(x=A, xt=0, w=B, wt=0, off=C, e=X, t=T, k=K, n=N, y=D, dx=1, dw=1, s=E, sb=saved, wk=F, wb=ws):
        return L.fp8_grouped_linear_forward(x, xt, w, wt, off, e, t, k, n, y, dx, dw, s, sb, wk, wb, None)

    assert fwd(xt=2) == ARG and fwd(wt=-1) == ARG and fwd(e=0) == SHAPE and fwd(e=513) == SHAPE
    assert fwd(t=-1) == SHAPE and fwd(n=1 << 21) == SHAPE and fwd(k=1 << 20, n=1 << 20, e=400) == SHAPE
    for missing in ("x", "w", "off", "y"):
        assert fwd(**{missing: None}) == ARG, missing
    assert fwd(x=A + 1) == ALIGN and fwd(off=C + 2) == ALIGN and fwd(wt=1, w=B + 2) == ALIGN
    assert fwd(s=None) == WS and fwd(sb=saved - 1) == WS and fwd(s=E + 16) == ALIGN
    assert fwd(wk=None) == WS and fwd(wb=100) == WS and fwd(wk=F + 16) == ALIGN

    def bwd(dy=A, xt=0, wt=0, off=C, e=X, t=T, k=K, n=N, dx=B, dw=D, s=E, sb=saved, wk=F, wb=ws):
        return L.fp8_grouped_linear_backward(dy, xt, wt, off, e, t, k, n, dx, dw, s, sb, wk, wb, None)

    assert bwd(dx=None, dw=None) == ARG and "both" in err(L)
    assert bwd(dy=None) == ARG and bwd(off=None) == ARG and bwd(xt=3) == ARG and bwd(k=-1) == SHAPE
    assert bwd(dx=B + 1) == ALIGN and bwd(wt=1, dw=D + 2) == ALIGN
    assert bwd(s=None) == WS and bwd(sb=saved - 1) == WS and bwd(wk=None) == WS and bwd(wb=1) == WS


def test_binding_refuses():
    f8 = lambda *s: torch.zeros(s, dtype=torch.float8_e4m3fn)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        fq.expert_order(i32(4, 2), 8)
    with pytest.raises(ValueError, match="device"):
        fq.fp8_grouped_gemm_b128(f8(4, 16), torch.zeros(1, 4), f8(2, 8, 16), torch.zeros(2, 1, 1), i32(3))
    with pytest.raises(ValueError, match="rows x in"):
        fq.fp8_grouped_linear(torch.zeros(4, 8), torch.zeros(2, 8, 9), i32(3))
    with pytest.raises(ValueError, match="device"):
        fq.fp8_grouped_linear(torch.zeros(4, 8), torch.zeros(2, 8, 8), i32(3))
