"""fp8_gemm_b128 where a product of two scales leaves binary32 and C does not.

The scales are powers of two and every sum is a few units of E4M3's smallest
products, so that C is exact."""
import pytest
import torch

import microscaling_fp4_quantization_amd as fq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROW, TILE = fq.B128_ROW, fq.B128_TILE

# m, n, k, type of C: at most 16 rows; 64, 128 and 256 tiles, with and without K ranges.
SHAPES = [(5, 300, 400, torch.float32), (5, 300, 400, torch.bfloat16), (90, 300, 400, torch.float32),
          (90, 300, 400, torch.bfloat16), (65, 517, 8208, torch.float32), (65, 517, 8208, torch.bfloat16),
          (1024, 4099, 144, torch.float32), (1024, 4099, 144, torch.bfloat16), (200, 4099, 4112, torch.float32),
          (200, 4099, 4112, torch.bfloat16), (2048, 4099, 400, torch.bfloat16), (4099, 1001, 4112, torch.bfloat16)]


def expected(a, sa, b, sb, kind):
    """C in binary64, block by block."""
    m, k = a.shape
    n = b.shape[0]
    c = torch.zeros(m, n, dtype=torch.float64, device=DEV)
    for s in range(sa.shape[0]):
        cols = slice(128 * s, min(k, 128 * s + 128))
        f = sb[:, s].double().repeat_interleave(128)[:n] if kind == TILE else sb[s].double()
        c += (a[:, cols].double() @ b[:, cols].double().t().contiguous()) * sa[s].double()[:, None] * f
    return c


@pytest.mark.parametrize("kind", [ROW, TILE])
@pytest.mark.parametrize("m,n,k,dtype", SHAPES)
def test_scale_products_past_the_range(m, n, k, dtype, kind):
    g = torch.Generator(device=DEV).manual_seed(m + n + k)
    pick = lambda *s: torch.randint(0, 6, s, generator=g, device=DEV)
    kb = -(-k // 128)
    # One element in ten is 2^-9 (E4M3's smallest) or its negative: sums of a few 2^-18 per block.
    def sparse(rows):
        v = torch.rand(rows, k, generator=g, device=DEV)
        return torch.where(v < 0.05, 2.0 ** -9, torch.where(v > 0.95, -(2.0 ** -9), 0.0))
    a, b = sparse(m), sparse(n)
    a[::7] = 0  # a row of zeros under large scales
    b[:, -1] = 2.0 ** -9
    # Products of 2^124 to 2^134, and in some rows over 2^180 under codes of zero.
    sa = torch.exp2(62.0 + pick(kb, m))
    sa[:, ::7] = 2.0 ** 120
    sb = torch.exp2(62.0 + pick(*((-(-n // 128), kb) if kind == TILE else (kb, n))))
    f8 = lambda x: x.to(torch.float8_e4m3fn)
    got = fq.fp8_gemm_b128(f8(a), sa, f8(b), sb, kind, dtype).double()
    want = expected(a, sa, b, sb, kind)
    # Below 2^128 a block's term is exact and the sum of kb of them rounds at each; a bf16 C rounds once more, and the
    # 8-bit matrix cores keep these products whole (they are all of one size).
    size = expected(a.abs(), sa, b.abs(), sb, kind)
    assert bool((size < 2.0 ** 127).all()) and bool((want[::7] == 0).all())
    err = (got - want).abs()
    assert bool((err <= (kb + 8) * 2.0 ** -23 * size + (2.0 ** -8 * want.abs() if dtype == torch.bfloat16 else 0)).all())


@pytest.mark.parametrize("m", [5, 90])
def test_row_scales_of_opposite_ends(m):
    """Scales of B near either end of the range, which A's bring back: the order of the factors is not seen."""
    n, k = 70, 128
    g = torch.Generator(device=DEV).manual_seed(3)
    ints = lambda r: torch.randint(-15, 16, (r, k), generator=g, device=DEV).float()
    for big in (118.0, -124.0):
        a, b = ints(m) * 2.0 ** -9, ints(n) * 2.0 ** -9
        if big > 0:
            a, b = a * 2.0 ** 13, b * 2.0 ** 13  # up to 240 each: sums of 2^22
        sa = torch.full((1, m), 2.0 ** -big, device=DEV)
        sb = torch.full((1, n), 2.0 ** big, device=DEV)
        f8 = lambda x: x.to(torch.float8_e4m3fn)
        got = fq.fp8_gemm_b128(f8(a), sa, f8(b), sb, ROW)
        assert torch.equal(got.double(), a.double() @ b.double().t().contiguous())


def test_quantize_takes_more_workgroups_than_a_grid_holds():
    """2^31 + 300 elements in one row, and in one column: 2^24 workgroups and some."""
    n = (1 << 31) + 300
    x = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    tail = torch.randn(300, device=DEV).to(torch.bfloat16)
    x[-300:] = tail
    want = fq.fp8_quantize_b128(tail.view(1, -1))
    q = fq.fp8_quantize_b128(x.view(1, -1))
    assert q.codes.shape == (1, n + 4)
    assert torch.equal(q.codes.view(torch.uint8)[:, -304:], want.codes.view(torch.uint8)) and torch.equal(q.scales[-3:], want.scales)
    assert not q.codes.view(torch.uint8)[:, :-304].any()
    del q
    q = fq.fp8_quantize_b128(x.view(-1, 1), codes=False, transposed=True)
    assert torch.equal(q.codes_t.view(torch.uint8)[:, -304:], want.codes.view(torch.uint8))
    assert torch.equal(q.scales_t[-3:], want.scales) and not q.codes_t.view(torch.uint8)[:, :-304].any()


def test_gemm_takes_more_workgroups_than_a_grid_holds():
    """2^30 + 70 rows of A: 2^24 + 2 tiles of 64.  Whole numbers: the last rows are exact."""
    m, n, k = (1 << 30) + 70, 8, 16
    g = torch.Generator(device=DEV).manual_seed(5)
    small = lambda r: torch.randint(-8, 9, (r, k), generator=g, device=DEV).float()
    tail, b = small(70), small(n)
    a = torch.zeros(m, k, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    a[-70:].view(torch.uint8).copy_(tail.to(torch.float8_e4m3fn).view(torch.uint8))
    one = lambda *s: torch.ones(*s, device=DEV)
    got = fq.fp8_gemm_b128(a, one(1, m), b.to(torch.float8_e4m3fn), one(1, 1))
    assert torch.equal(got[-70:].double(), tail.double() @ b.double().t().contiguous())
    assert not got[:-70].any()
