"""int8_gemm's large tiles, whole and in quarters, and its K ranges, each at the scales, outputs and
biases where it can go wrong; test_tile_choice.py holds that the shapes take the kernels that they
are here for.  Expectations as in test_gpu_int8.py: equal bit for bit without a bias."""
import pytest
import torch

import microscaling_fp4_quantization_amd as fq
from test_gpu_int8 import TYPES, expect, gen, operands, product

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# (M, N, K): (tile, K ranges, quartered tiles).  C's rows start on 16 bytes in the second and the
# third, end inside 16 bytes in the others.
LARGE = {(4100, 4099, 1040): (256, 1, 33), (4096, 4096, 4096): (256, 1, 0), (4400, 4104, 4096): (256, 1, 50)}
# Blocks of K that do not divide into the ranges, a last block of 16, N odd and N % 4 == 2, one row
# of tiles only.
RANGES = {(1024, 3584, 18944): (256, 4, 0), (2048, 3584, 18944): (256, 2, 0), (1024, 3585, 18960): (256, 4, 0), (500, 3001, 18960): (256, 8, 0),
          (512, 3584, 18944): (128, 4, 0), (2000, 1003, 18960): (128, 4, 0), (1020, 1030, 16016): (128, 6, 0), (700, 1003, 9008): (64, 4, 0)}


def any_scales(m, n, seed):
    """Scales from 2^-126 to 2^126, most pairs with a product that is no normal number."""
    g = gen(seed)
    scale = lambda r: torch.exp2(torch.randint(-126, 127, (r,), generator=g, device=DEV).float())
    return scale(m), scale(n) * 1.25


def by_range(acc, sa, sb):
    """The rounded form where sa sb is a normal number, elsewhere the exact one (24 + 24 bits and a power of two)."""
    f = sa[:, None] * sb
    normal = (f.abs() >= 2.0 ** -126) & torch.isfinite(f)
    return torch.where(normal, expect(acc, sa, sb), acc * (sa.double()[:, None] * sb.double())).float()


@pytest.mark.parametrize("m,n,k", [*LARGE, *RANGES])
def test_scales_of_any_size(m, n, k):
    a, sa, b, sb = operands(m, n, k, 11)
    acc = product(a, b)
    for s, t in (any_scales(m, n, 12), (sa, sb)):
        want = by_range(acc, s, t)
        assert torch.equal(fq.int8_gemm(a, s, b, t), want)
        assert torch.equal(fq.int8_gemm(a, s, b, t, out_dtype=torch.bfloat16), want.bfloat16())
    # One row and one column alone: their tiles take the full form, the others the plain one.
    sa[m - 2], sb[n // 2] = 2.0 ** -120, 2.0 ** 125
    want = by_range(acc, sa, sb)
    assert torch.equal(fq.int8_gemm(a, sa, b, sb), want)
    assert torch.equal(fq.int8_gemm(a, sa, b, sb, out_dtype=torch.bfloat16), want.bfloat16())


@pytest.mark.parametrize("m,n,k", [*LARGE, *RANGES])
def test_scales_that_are_not_finite(m, n, k):
    a, sa, b, sb = operands(m, n, k, 13)
    a[1], b[3] = 0, 0  # as the quantizer leaves such rows
    sa[m - 1], sa[1], sb[3] = float("nan"), float("inf"), float("inf")
    for dtype in TYPES:
        c = fq.int8_gemm(a, sa, b, sb, out_dtype=dtype)
        assert bool(c[m - 1].isnan().all()) and bool(c[1].isnan().all()) and bool(c[:, 3].isnan().all())
        rows, cols = torch.ones(m, dtype=torch.bool, device=DEV), torch.ones(n, dtype=torch.bool, device=DEV)
        rows[1], rows[m - 1], cols[3] = False, False, False
        assert torch.equal(c[rows][:, cols], by_range(product(a, b), sa, sb).to(dtype)[rows][:, cols])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", [*LARGE, *RANGES])
def test_bias(m, n, k, dtype):
    """Half a step of the value formed in 64 bits; scales of any size too, in binary64 before one rounding."""
    a, sa, b, sb = operands(m, n, k, 5)
    acc = product(a, b)
    bias = torch.randn(n, generator=gen(6), device=DEV).to(dtype) * 100
    for s, t in ((sa, sb), any_scales(m, n, 7)):
        f = s[:, None] * t
        normal = (f >= 2.0 ** -126) & torch.isfinite(f)
        want = torch.where(normal, expect(acc, s, t, bias), acc * (s.double()[:, None] * t.double()) + bias.double())
        got = fq.int8_gemm(a, s, b, t, bias)
        inside = want.abs() < 2.0 ** 127.9
        assert bool(((got.double() - want).abs() <= 2.0 ** -24 * (1 + 2.0 ** -20) * want.abs() + 2.0 ** -149)[inside].all())
        assert torch.equal(fq.int8_gemm(a, s, b, t, bias, out_dtype=torch.bfloat16), got.bfloat16())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", [*LARGE, *RANGES])
def test_outputs_on_any_element(m, n, k, dtype):
    a, sa, b, sb = operands(m, n, k, 17)
    buf = torch.full((m * n + 3,), 7.0, dtype=dtype, device=DEV)
    out = buf[1:1 + m * n].view(m, n)
    fq.int8_gemm(a, sa, b, sb, out=out)
    assert torch.equal(out, expect(product(a, b), sa, sb).float().to(dtype))
    assert buf[0] == 7.0 and bool((buf[1 + m * n:] == 7.0).all())


@pytest.mark.parametrize("m,n,k", RANGES)
def test_ranges_write_their_workspace_alone(m, n, k):
    """Sums of the largest codes, through a workspace of the exact size."""
    a, sa, b, sb = operands(m, n, k, 9, extreme=True)
    need = fq.lib().int8_gemm_workspace_bytes(m, n, k)
    ws = torch.full((need + 512,), 9, dtype=torch.uint8, device=DEV)
    c = fq.int8_gemm(a, sa, b, sb, ws=ws[256:256 + need])
    acc = torch.full((m, n), 2.0 ** 14 * k, dtype=torch.float64, device=DEV)
    assert torch.equal(c, expect(acc, sa, sb).float())
    assert bool((ws[:256] == 9).all()) and bool((ws[256 + need:] == 9).all())


@pytest.mark.parametrize("m,n,k", [(4100, 4099, 1040), (1024, 3585, 18960), (2000, 1003, 18960)])
def test_a_token_among_others_and_alone(m, n, k):
    a, sa, b, sb = operands(m, n, k, 21)
    bias = torch.randn(n, generator=gen(22), device=DEV)
    whole = fq.int8_gemm(a, sa, b, sb, bias)
    for lo, hi in ((0, 1), (m - 20, m - 3), (100, 190), (m - 1, m)):
        assert torch.equal(fq.int8_gemm(a[lo:hi], sa[lo:hi], b, sb, bias), whole[lo:hi])


MORE = [(1, 300, 512), (16, 511, 4096), (333, 1031, 1008), (4100, 4099, 384)]  # few rows, tiles of 64 and 128


@pytest.mark.parametrize("m,n,k", [*MORE, *LARGE, *RANGES])
def test_padding(m, n, k):
    """Rows and columns of zeros, as a padded batch and dropped channels leave them (scale 2^-126, every
    product of scales below the range), and elsewhere codes that are not 0 under such a scale."""
    a, sa, b, sb = operands(m, n, k, 31)
    sa.clamp_(max=0.5)
    for row in (m // 3, *range(max(m - 70, 0), m)):
        a[row], sa[row] = 0, 2.0 ** -126
    b[n // 2], sb[n // 2], b[n - 1], sb[n - 1] = 0, 2.0 ** -126, 0, 2.0 ** -126
    bias = torch.randn(n, generator=gen(32), device=DEV)
    for tiny in (False, True):
        if tiny:
            a[m // 2].fill_(1)
            sa[m // 2] = 2.0 ** -126
        acc = product(a, b)
        want = by_range(acc, sa, sb)
        assert torch.equal(fq.int8_gemm(a, sa, b, sb), want)
        assert torch.equal(fq.int8_gemm(a, sa, b, sb, out_dtype=torch.bfloat16), want.bfloat16())
        full = acc * (sa.double()[:, None] * sb.double()) + bias.double()
        got = fq.int8_gemm(a, sa, b, sb, bias)
        assert bool(((got.double() - full).abs() <= 2.0 ** -24 * (full.abs() + 2 * (full - bias.double()).abs()) * (1 + 2.0 ** -20)).all())
        zero = (acc == 0)
        assert torch.equal(got[zero], bias.expand(m, n)[zero])
        if tiny and m // 2 == m // 3:
            break  # (one row alone: it is not of zeros any more)
        sa[m // 3] = float("inf")  # zeros under an infinite scale are NaN, whatever the other rows are
        assert bool(fq.int8_gemm(a, sa, b, sb, bias)[m // 3].isnan().all())
        sa[m // 3] = 2.0 ** -126


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,k,n", [(40, 200, 300), (600, 2048, 5000), (4100, 1040, 4099)])
def test_linear_of_a_padded_batch(tokens, k, n, dtype):
    """A batch padded with rows of zeros: its own tokens' bits, and the bias in the others."""
    g = gen(tokens)
    x = torch.randn(tokens, k, generator=g, device=DEV).to(dtype)
    w = fq.int8_quantize_rows(torch.randn(n, k, generator=g, device=DEV) * 0.05)
    bias = torch.randn(n, generator=g, device=DEV).to(dtype)
    real = tokens * 2 // 3
    want = fq.int8_linear(x[:real], w, bias)
    x[real:] = 0
    y = fq.int8_linear(x, w, bias)
    assert torch.equal(y[:real], want) and torch.equal(y[real:], bias.expand(tokens - real, n))
