"""The grouped kernels of large steps: each tile of y, dx and dw, each with scales whose product
passes binary32's range and with NaN; test_tile_choice.py holds that the shapes take the kernels
that they are here for.  Bounds as in test_gpu_grouped.py."""
import pytest
import torch

import microscaling_fp4_quantization_amd as fq
from test_gpu_grouped import DEV, ROW, TILE, TYPES, bar, expect, experts_of, gen, i32, linear_expect, sizes_to_ends, value

pytestmark = pytest.mark.gpu

BF16, F32 = TYPES
# Sizes of the groups, N, K: (tiles of y, dx and dw in bf16, in binary32).  Unequal groups of many
# blocks, none, one of a single row, two of one size, and more than 64 experts.
STEPS = [(([3000, 0, 1700, 2500, 5000, 1100], 2048, 2048), (256, 256, 256), (128, 128, 128)),
         (([3000, 0, 1701, 2500, 5000, 1, 901], 2200, 2064), (256, 256, 256), (128, 128, 128)),
         (([3000, 0, 1701, 2500, 5000, 1, 1701], 2200, 2064), (128, 128, 256), (128, 128, 128)),
         (([3000, 0, 1700, 2500], 1400, 1100), (256, 256, 128), (128, 128, 128)),
         (([1500, 0, 900], 2048, 2047), (128, 128, 256), (128, 128, 128)),
         (([0, 130] * 35, 1000, 1100), (64, 64, 256), (64, 64, 128))]


@pytest.mark.parametrize("xt", TYPES)
@pytest.mark.parametrize("wt", TYPES)
@pytest.mark.parametrize("sizes,n,k", [s[0] for s in STEPS])
def test_linear(sizes, n, k, xt, wt):
    g = gen(n + k)
    ends = sizes_to_ends(sizes)
    rows = ends[-1] + 5
    x = torch.randn(rows, k, generator=g, device=DEV).to(xt).requires_grad_()
    w = (torch.randn(len(sizes), n, k, generator=g, device=DEV) * 0.1).to(wt).requires_grad_()
    dy = (torch.randn(rows, n, generator=g, device=DEV) * 1e-2).to(xt)
    y = fq.fp8_grouped_linear(x, w, i32(ends))
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    want = linear_expect(x.detach(), w.detach(), dy, ends)
    for name, got, terms in (("y", y.detach(), k), ("dx", dx, n), ("dw", dw, max(sizes))):
        v, size = want[name]
        err, lim = (got.double() - v).abs(), bar(v, size, terms, got.dtype)
        assert bool((err <= lim).all()), (name, float((err / lim).nan_to_num().max()))
    assert bool((y[ends[-1]:] == 0).all()) and bool((dx[ends[-1]:] == 0).all())
    for e, m in enumerate(sizes):
        assert m or bool((dw[e] == 0).all())
    again = torch.autograd.grad(fq.fp8_grouped_linear(x, w, i32(ends)), (x, w), dy)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes,n,k", [([100, 0, 300], 200, 136), STEPS[0][0], STEPS[3][0], STEPS[4][0]])
def test_weight_gradient_of_scale_products_past_the_range(sizes, n, k, dtype):
    """In each block of 128 rows x is 448 2^64 in one, where dy is 0, and dy in another, where x is
    0; elsewhere both are 2^55: scales of 2^64 each, codes of 2^-9, sums below 2^127."""
    g = gen(n)
    ends = sizes_to_ends(sizes)
    rows = ends[-1]
    sign = lambda *s: torch.randint(0, 2, s, generator=g, device=DEV).float() * 2 - 1
    x, dy = sign(rows, k) * 2.0 ** 55, sign(rows, n) * 2.0 ** 55
    for lo, hi in zip(ends, ends[1:]):
        for b in range(lo, hi, 128):
            if hi - b > 1:
                x[b], dy[b] = 448 * 2.0 ** 64, 0.0
                x[b + 1], dy[b + 1] = 0.0, 448 * 2.0 ** 64
    x, dy = x.to(dtype), dy.to(dtype)
    w = (torch.randn(len(sizes), n, k, generator=g, device=DEV) * 2.0 ** -90).to(dtype).requires_grad_()
    dw, = torch.autograd.grad(fq.fp8_grouped_linear(x, w, i32(ends)), w, dy)
    v, size = linear_expect(x, w.detach(), dy, ends)["dw"]
    assert bool((size < 2.0 ** 127).all()) and bool((v.abs() > 2.0 ** 110).any())
    assert bool(((dw.double() - v).abs() <= bar(v, size, max(sizes), dtype)).all())


# Sizes, N, K of the product: the tile in bf16 and in binary32.
PRODUCTS = [(([3000, 0, 1700, 2500, 5000], 2048, 2048), 256, 128), (([3000, 0, 1701, 2500, 5000], 2200, 2064), 256, 128),
            (([1000, 0, 1400], 2048, 2048), 128, 128)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("form", ["experts", "stacked", "gathered"])
@pytest.mark.parametrize("sizes,n,k", [p[0] for p in PRODUCTS])
def test_scale_products_past_the_range(sizes, n, k, form, dtype):
    """Scales of 2^62 and more under codes whose products are exact and small enough."""
    g = gen(n)
    e, ends = len(sizes), sizes_to_ends(sizes)
    rows = ends[-1] + 3
    up = lambda v: -(-v // 128)

    def sparse(*s):
        v = torch.rand(*s, generator=g, device=DEV)
        return torch.where(v < 0.05, 2.0 ** -9, torch.where(v > 0.95, -(2.0 ** -9), 0.0)).to(torch.float8_e4m3fn)

    pick = lambda *s: torch.exp2(62.0 + torch.randint(0, 6, s, generator=g, device=DEV))
    a_rows = 1000 if form == "gathered" else rows
    a, sa = sparse(a_rows, k), pick(up(k), a_rows)
    tokens = torch.randint(0, a_rows, (rows,), generator=g, device=DEV, dtype=torch.int32) if form == "gathered" else None
    if form == "stacked":
        b, sb = sparse(e * n, k), pick(up(e * n), up(k))
        wv = value(b, sb, TILE).view(e, n, k)
    else:
        b, sb = sparse(e, n, k), pick(e, up(n), up(k))
        wv = torch.stack([value(c, s, TILE) for c, s in zip(b, sb)])
    out = torch.full((rows, n), 77.0, dtype=dtype, device=DEV)
    fq.fp8_grouped_gemm_b128(a, sa, b, sb, i32(ends), tokens=tokens, out=out)
    want, size = expect(value(a, sa, ROW), wv, ends, tokens, rows)
    assert bool((size[:ends[-1]] < 2.0 ** 127).all()) and bool((out[ends[-1]:] == 77.0).all())
    lim = (up(k) + 8) * 2.0 ** -23 * size + (2.0 ** -8 * want.abs() if dtype == BF16 else 0)
    assert bool(((out.double() - want).abs() <= lim)[:ends[-1]].all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("form", ["experts", "gathered"])
@pytest.mark.parametrize("sizes,n,k", [p[0] for p in PRODUCTS])
def test_nan_stays_in_its_rows_and_columns(sizes, n, k, form, dtype):
    g = gen(k)
    ends = sizes_to_ends(sizes)
    rows = ends[-1]
    codes, scales = experts_of(torch.randn(len(sizes), n, k, generator=g, device=DEV))
    qa = fq.fp8_quantize_b128(torch.randn(rows, k, generator=g, device=DEV))
    tokens = torch.randperm(rows, generator=g, device=DEV).int() if form == "gathered" else torch.arange(rows, device=DEV).int()
    call = lambda: fq.fp8_grouped_gemm_b128(qa.codes, qa.scales, codes, scales, i32(ends), tokens=tokens if form == "gathered" else None,
                                            out_dtype=dtype)
    want = call()
    bad = [1, rows - 700]  # rows of A: a code and a scale
    qa.codes.view(torch.uint8)[bad[0], k - 1] = 0x7F
    qa.scales[1, bad[1]] = float("nan")
    scales[2, 1, 0] = float("nan")  # columns 128 .. 255 of group 2
    got = call()
    keep = torch.ones(rows, n, dtype=torch.bool, device=DEV)
    for row in bad:
        keep[tokens == row] = False
    keep[ends[2]:ends[3], 128:256] = False
    assert torch.equal(got[keep], want[keep]) and bool(got[~keep].isnan().all())


# Sizes, N, K; N is no multiple of 128, so that experts start inside a block of the stacked scales.
# The pass over the weights, tiles of 64, of 128, of 256 in bf16.
STACKED = [(([3, 0, 16, 1], 48, 400), 0, 0), (([128, 129, 0, 127], 200, 512), 64, 64), (([1000, 0, 1400], 2040, 2048), 128, 128),
           (([3000, 0, 1701, 2500, 5000], 2200, 2064), 256, 128)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("large_scales", [False, True])
@pytest.mark.parametrize("sizes,n,k", [s[0] for s in STACKED])
def test_stacked_scales_and_gathered_rows(sizes, n, k, large_scales, dtype):
    g = gen(n + 1)
    e, ends = len(sizes), sizes_to_ends(sizes)
    rows, a_rows, up = ends[-1] + 3, ends[-1] // 2 + 1, lambda v: -(-v // 128)
    if large_scales:  # as in test_scale_products_past_the_range
        few = lambda *s: (torch.randint(-9, 10, s, generator=g, device=DEV).div(9, rounding_mode="trunc") * 2.0 ** -9).to(torch.float8_e4m3fn)
        pick = lambda *s: torch.exp2(62.0 + torch.randint(0, 6, s, generator=g, device=DEV))
        a, sa, b, sb = few(a_rows, k), pick(up(k), a_rows), few(e * n, k), pick(up(e * n), up(k))
    else:
        qa = fq.fp8_quantize_b128(torch.randn(a_rows, k, generator=g, device=DEV))
        qb = fq.fp8_quantize_b128(torch.randn(e * n, k, generator=g, device=DEV), TILE)
        a, sa, b, sb = qa.codes, qa.scales, qb.codes, qb.scales
    tokens = torch.randint(-1, a_rows + 1, (rows,), generator=g, device=DEV, dtype=torch.int32)  # some that A does not have
    out = torch.full((rows, n), 77.0, dtype=dtype, device=DEV)
    fq.fp8_grouped_gemm_b128(a, sa, b, sb, i32(ends), tokens=tokens, out=out)
    av = torch.cat([value(a, sa, ROW), torch.zeros(1, a.shape[1], dtype=torch.float64, device=DEV)])
    want, size = expect(av, value(b, sb, TILE).view(e, n, -1), ends, torch.where((tokens >= 0) & (tokens < a_rows), tokens, a_rows), rows)
    assert bool((size[:ends[-1]] < 2.0 ** 127).all()) and bool((out[ends[-1]:] == 77.0).all())
    assert bool(((out.double() - want).abs() <= bar(want, size, k, dtype))[:ends[-1]].all())
    # NaN stays in its rows, and in its expert's columns.
    some = int(tokens[ends[2]].clamp(0, a_rows - 1))
    sa[0, some], b.view(torch.uint8)[2 * n + 5, 7] = float("nan"), 0x7F
    got = fq.fp8_grouped_gemm_b128(a, sa, b, sb, i32(ends), tokens=tokens, out=torch.full_like(out, 77.0))
    bad = (tokens == some)[:, None].expand(rows, n).clone()
    bad[ends[2]:ends[3], 5] = True
    bad[ends[-1]:] = False
    assert bool(got[bad].isnan().all()) and torch.equal(got[~bad], out[~bad])
