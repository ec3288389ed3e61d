"""fp8_gemm_b128 at shapes that take each of its kernels, against 64 bits.

The bars are those of the product's other tests: (K/128 + 8) 2^-23 S for a binary32
C and 2^-14 S + 2^-8 |C| for a bf16 one, S = |A_hat| |B_hat|^T.  Every element is
compared; the reference is a binary64 product of the stored operands.
"""
import pytest
import torch

import microscaling_fp4_quantization_amd as fq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROW, TILE = fq.B128_ROW, fq.B128_TILE
BF16, F32 = torch.bfloat16, torch.float32


def operand(rows, k, kind, seed):
    """Codes and scales of Normal values of a wide spread per row, and their binary64 values."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(rows, k, generator=g, device=DEV)
    x *= torch.exp2(torch.randint(-3, 4, (rows, 1), generator=g, device=DEV).float())
    q = fq.fp8_quantize_b128(x, kind)
    return q.codes, q.scales, value(q.codes, q.scales, kind)


def value(codes, scales, kind):
    r, c = (torch.arange(n, device=DEV) for n in codes.shape)
    s = scales.double()[r // 128] if kind == TILE else scales.double().t()
    return codes.float().double() * s[:, c // 128]


def ranges(m, n, k, dtype):
    """K ranges that the library takes, by the workspace that it asks for."""
    return max(1, fq.lib().fp8_gemm_b128_workspace_bytes(m, n, k, fq.F32 if dtype == F32 else fq.BF16) // (4 * m * n))


# m, n, k, type of C, K ranges; the kernel that the shape takes.  K ends inside a block of 128
# and C's rows end inside 16 bytes in every group.
KERNELS = [
    (16, 333, 1040, F32, 1),      # at most 16 rows
    (300, 1001, 1008, F32, 1),    # 64 x 64
    (300, 1001, 1008, BF16, 1),
    (65, 517, 8208, F32, 8),      # 64 x 64, K ranges
    (65, 517, 8208, BF16, 8),
    (1024, 4099, 144, F32, 1),    # 128 x 128
    (1024, 4099, 144, BF16, 1),
    (200, 14336, 896, BF16, 1),
    (200, 4099, 4112, F32, 3),    # 128 x 128, K ranges
    (200, 4099, 4112, BF16, 3),
    (100, 3584, 14336, BF16, 8),
    (2048, 4099, 400, BF16, 1),   # 256 x 256
    (515, 14336, 272, BF16, 1),
    (4099, 1001, 4112, BF16, 3),  # 256 x 256, K ranges
    (200, 8192, 14336, BF16, 8),
]


@pytest.mark.parametrize("kind", [ROW, TILE])
@pytest.mark.parametrize("m,n,k,dtype,split", KERNELS)
def test_each_kernel_within_bound(m, n, k, dtype, split, kind):
    assert ranges(m, n, k, dtype) == split
    a, sa, av = operand(m, k, ROW, 1)
    b, sb, bv = operand(n, k, kind, 2)
    got = fq.fp8_gemm_b128(a, sa, b, sb, kind, dtype).double()
    want, size = av @ bv.t().contiguous(), av.abs() @ bv.abs().t().contiguous()
    bar = (k / 128 + 8) * 2.0 ** -23 * size if dtype == F32 else 2.0 ** -14 * size + 2.0 ** -8 * want.abs()
    err = (got - want).abs()
    assert bool((err <= bar).all()), float((err / bar).max())


@pytest.mark.parametrize("kind", [ROW, TILE])
@pytest.mark.parametrize("m,n,k,dtype,split", KERNELS)
def test_each_kernel_keeps_a_nan_where_it_belongs(m, n, k, dtype, split, kind):
    """A NaN code of A and one of B, a NaN scale of each: their rows and columns are NaN, the rest is as without."""
    a, sa, _ = operand(m, k, ROW, 3)
    b, sb, _ = operand(n, k, kind, 4)
    clean = fq.fp8_gemm_b128(a, sa, b, sb, kind, dtype)
    a.view(torch.uint8)[m - 1, k - 1] = 0x7F
    b.view(torch.uint8)[1, 5] = 0xFF
    sa[0, 2] = float("nan")
    if kind == TILE:
        sb[(n - 1) // 128, -1] = float("nan")
    else:
        sb[-1, n - 3] = float("nan")
    got = fq.fp8_gemm_b128(a, sa, b, sb, kind, dtype)
    hit = torch.zeros(m, n, dtype=torch.bool, device=DEV)
    hit[[2, m - 1]] = True
    hit[:, 1] = True
    if kind == TILE:
        hit[:, (n - 1) // 128 * 128:] = True
    else:
        hit[:, n - 3] = True
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit])
