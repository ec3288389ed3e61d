"""The 8-bit block-128 quantizer, product and linear layer against their
definitions in 64 bits.

Bars, from the arithmetic:
 - codes and scales: every operation of the definition is a correctly rounded one,
   so they are equal, bit for bit;
 - product: each block's 128 products (exact in binary32, at most 8 significant
   bits) are added from zero by the matrix cores, the scales' product and each
   fused multiply-add round once, K ranges meet in binary64.  Each rounding is at
   most 2^-24 of a partial sum, which |A_hat| |B_hat|^T bounds: K/128 of them
   along K and under 8 within a block, with a factor 2 of headroom:
   (K/128 + 8) 2^-23 |A_hat| |B_hat|^T.  A bf16 output is one rounding to nearest
   (half an ulp, 2^-9 |C|, with the same headroom) of sums that may come from the
   8-bit matrix cores, which keep a product to about 2^-17 of the largest in its
   sum: 2^-15.5 of sum |a b| at most over Normal operands (measured on the
   instruction alone).  It has 2^-8 |C| + 2^-14 |A_hat| |B_hat|^T;
 - where every partial sum is a whole number below 2^24 and the scales are 1, the
   product is exact.
"""
import numpy as np
import pytest
import torch

import fp8_ref as ref
import microscaling_fp4_quantization_amd as fq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROW, TILE = fq.B128_ROW, fq.B128_TILE


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def codes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def values(rows, cols, seed, dtype):
    """Normal values of a wide spread, blocks of zeros, single values, denormals and -0 among them."""
    rng = np.random.default_rng([seed, rows, cols])
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-6, 7, (rows, 1)).astype(float))
    x[rng.random((rows, cols)) < 0.02] = 0.0
    x[rng.random((rows, cols)) < 0.02] = -0.0
    if rows > 3:
        x[1] = 0.0
        x[2, cols // 2:] *= 1e-40
        x[3] *= 1e30
    t = torch.from_numpy(x.astype(np.float32)).to(dtype)
    return t, t.float().numpy()


SIZES = [(1, 1), (1, 16), (1, 128), (3, 127), (2, 129), (127, 8), (128, 128), (129, 130), (130, 1000), (257, 96),
         (64, 896), (300, 17), (5, 4097)]


@pytest.mark.parametrize("kind", [ROW, TILE])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize_is_the_definition(rows, cols, dtype, kind):
    t, x = values(rows, cols, 1, dtype)
    q = fq.fp8_quantize_b128(t.to(DEV), kind, transposed=True)
    for got_c, got_s, src in ((q.codes, q.scales, x), (q.codes_t, q.scales_t, x.T)):
        c, s = ref.quantize(src, kind == TILE)
        np.testing.assert_array_equal(got_s.cpu().numpy(), s)
        np.testing.assert_array_equal(codes_of(got_c), c)


@pytest.mark.parametrize("kind", [ROW, TILE])
@pytest.mark.parametrize("rows,cols", [(130, 200), (1, 129), (256, 384)])
def test_each_output_alone_is_the_same(rows, cols, kind):
    x = values(rows, cols, 2, torch.bfloat16)[0].to(DEV)
    both = fq.fp8_quantize_b128(x, kind, transposed=True)
    a = fq.fp8_quantize_b128(x, kind)
    b = fq.fp8_quantize_b128(x, kind, codes=False, transposed=True)
    assert a.codes_t is None and b.codes is None
    np.testing.assert_array_equal(codes_of(a.codes), codes_of(both.codes))
    np.testing.assert_array_equal(codes_of(b.codes_t), codes_of(both.codes_t))
    assert torch.equal(a.scales, both.scales) and torch.equal(b.scales_t, both.scales_t)


@pytest.mark.parametrize("e", [-149, -140, -126, -100, -62, -60, -58, 0, 60, 99, 101, 119])
def test_scales_over_the_whole_exponent_range(e):
    """Every scale from the floor to the largest, both sides of the corrected quotient's range."""
    rng = np.random.default_rng(e + 200)
    x = np.ldexp(rng.uniform(1, 2, (6, 128)) * rng.choice([-1, 1], (6, 128)), e + rng.integers(-12, 8, (6, 128)))
    x = x.astype(np.float32)
    q = fq.fp8_quantize_b128(dev(x), ROW, transposed=True)
    c, s = ref.quantize(x, False)
    np.testing.assert_array_equal(q.scales.cpu().numpy(), s)
    np.testing.assert_array_equal(codes_of(q.codes), c)
    c, s = ref.quantize(x.T, False)
    np.testing.assert_array_equal(q.scales_t.cpu().numpy(), s)
    np.testing.assert_array_equal(codes_of(q.codes_t), c)


def test_quantize_ties_go_to_the_even_code():
    mids = (ref.VALUES[:-1] + ref.VALUES[1:]) / 2
    x = np.zeros((2, 128), np.float32)
    x[0, :126], x[1, :126] = mids, -mids
    x[:, 127] = 448.0  # scale 1
    q = fq.fp8_quantize_b128(dev(x))
    assert torch.equal(q.scales.cpu(), torch.ones(1, 2))
    even = np.array([c if c % 2 == 0 else c + 1 for c in range(126)], np.uint8)
    np.testing.assert_array_equal(codes_of(q.codes)[0, :126], even)
    np.testing.assert_array_equal(codes_of(q.codes)[1, :126], even | 0x80)


@pytest.mark.parametrize("offset", [1, 2, 3, 5])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_reads_any_alignment(dtype, offset):
    rows, cols = 37, 200
    t, x = values(rows, cols, 3, dtype)
    flat = torch.zeros(rows * cols + offset, dtype=dtype, device=DEV)
    flat[offset:] = t.to(DEV).flatten()
    q = fq.fp8_quantize_b128(flat[offset:].view(rows, cols), ROW, transposed=True)
    np.testing.assert_array_equal(codes_of(q.codes), ref.quantize(x, False)[0])
    np.testing.assert_array_equal(codes_of(q.codes_t), ref.quantize(x.T, False)[0])


@pytest.mark.parametrize("rows,cols", [(0, 5), (5, 0), (0, 0)])
def test_quantize_of_nothing(rows, cols):
    q = fq.fp8_quantize_b128(torch.zeros(rows, cols, device=DEV), ROW, transposed=True)
    assert q.codes.shape == (rows, -(-cols // 16) * 16) and q.codes_t.shape == (cols, -(-rows // 16) * 16)


def operand(rows, k, seed, tile):
    rng = np.random.default_rng([seed, rows, k])
    x = (rng.standard_normal((rows, k)) * np.exp2(rng.integers(-3, 4, (rows, 1)).astype(float))).astype(np.float32)
    return ref.quantize(x, tile)


def product(a, b, kind, out_dtype=torch.float32):
    f8 = lambda c: dev(c).view(torch.float8_e4m3fn)
    return fq.fp8_gemm_b128(f8(a[0]), dev(a[1]), f8(b[0]), dev(b[1]), kind, out_dtype).float().cpu().numpy()


# Both kernels and each of their sizes: few rows (1..16, 17..32, 33..64), tiles
# (with and without K ranges), K blocks cut short, columns that are no whole 16 bytes.
SHAPES = [(1, 1, 16), (1, 16, 128), (2, 17, 144), (16, 300, 256), (17, 33, 384), (31, 96, 1008), (33, 100, 128),
          (64, 257, 2064), (5, 1000, 4096), (65, 64, 128), (66, 70, 16), (130, 300, 272), (256, 256, 256),
          (257, 129, 1008), (300, 517, 1152), (200, 333, 4112), (777, 1031, 640), (70, 8, 8192), (1, 4100, 512)]


@pytest.mark.parametrize("kind", [ROW, TILE])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm_within_bound(m, n, k, kind):
    a, b = operand(m, k, 4, False), operand(n, k, 5, kind == TILE)
    av, bv = ref.value(*a, False), ref.value(*b, kind == TILE)
    want, size = av @ bv.T, np.abs(av) @ np.abs(bv).T
    tol = (k / 128 + 8) * 2.0 ** -23 * size
    for dt, bar in ((torch.float32, tol), (torch.bfloat16, 2.0 ** -14 * size + 2.0 ** -8 * np.abs(want))):
        err = np.abs(product(a, b, kind, dt) - want)
        assert np.all(err <= bar), (dt, np.max(err / bar))


@pytest.mark.parametrize("kind", [ROW, TILE])
@pytest.mark.parametrize("m,n,k", [(1, 40, 256), (40, 24, 400), (64, 128, 128), (100, 300, 256), (300, 260, 528)])
def test_gemm_exact_on_whole_numbers(m, n, k, kind):
    rng = np.random.default_rng([6, m, n, k])
    av, bv = rng.integers(-8, 9, (m, k)).astype(float), rng.integers(-8, 9, (n, k)).astype(float)
    kb = k // 128 + (k % 128 > 0)
    ones = lambda rows, tile: np.ones((-(-rows // 128), kb) if tile else (kb, rows), np.float32)
    a, b = (ref.to_codes(av), ones(m, False)), (ref.to_codes(bv), ones(n, kind == TILE))
    np.testing.assert_array_equal(product(a, b, kind), av @ bv.T)


@pytest.mark.parametrize("kind", [ROW, TILE])
@pytest.mark.parametrize("m", [3, 100])
def test_gemm_scales_meet_their_own_blocks(m, kind):
    """Codes of ones, every scale its own power of two: each block's share is told apart, exactly."""
    n, k = 300, 384
    rng = np.random.default_rng(7)
    sa = np.exp2(rng.integers(-3, 3, (3, m))).astype(np.float32)
    sb = np.exp2(rng.integers(-3, 3, (3, 3) if kind == TILE else (3, n))).astype(np.float32)
    one = lambda rows: ref.to_codes(np.ones((rows, k)))
    got = product((one(m), sa), (one(n), sb), kind)
    full = sb[np.arange(n) // 128] if kind == TILE else sb.T
    np.testing.assert_array_equal(got, 128.0 * sa.T.astype(float) @ full.T.astype(float))


@pytest.mark.parametrize("m", [2, 90])
def test_gemm_keeps_a_nan_in_its_row(m):
    k, n = 256, 140
    a, b = operand(m, k, 8, False), operand(n, k, 9, True)
    a[0][1, 130] = 0x7F
    got = product(a, b, TILE)
    assert np.isnan(got[1]).all() and np.isfinite(np.delete(got, 1, 0)).all()


def test_gemm_of_nothing():
    z = lambda *s: torch.zeros(*s, device=DEV)
    f8 = lambda *s: z(*s).to(torch.float8_e4m3fn)
    assert fq.fp8_gemm_b128(f8(0, 32), z(1, 0), f8(5, 32), z(1, 1)).shape == (0, 5)
    for m in (3, 100):
        out = torch.full((m, 5), 7.0, device=DEV)
        fq.fp8_gemm_b128(f8(m, 0), z(0, m), f8(5, 0), z(1, 0), TILE, out=out)
        assert torch.equal(out, torch.zeros_like(out))


def test_gemm_refusals():
    a, sa = torch.zeros(4, 32, device=DEV).to(torch.float8_e4m3fn), torch.zeros(1, 4, device=DEV)
    b, sb = torch.zeros(6, 32, device=DEV).to(torch.float8_e4m3fn), torch.zeros(1, 1, device=DEV)
    with pytest.raises(ValueError, match="scales"):
        fq.fp8_gemm_b128(a, sa, b, sb, ROW)
    with pytest.raises(ValueError, match="scales"):
        fq.fp8_gemm_b128(a, sa.t().contiguous(), b, sb)
    with pytest.raises(TypeError):
        fq.fp8_gemm_b128(a.view(torch.uint8), sa, b, sb)
    with pytest.raises(ValueError, match="contiguous"):
        fq.fp8_gemm_b128(a.t(), sa, b, sb)
    with pytest.raises(ValueError, match="rows of"):
        fq.fp8_gemm_b128(a, sa, b[:, :16].contiguous(), sb)
    with pytest.raises(ValueError, match="b_kind"):
        fq.fp8_gemm_b128(a, sa, b, sb, 2)
    with pytest.raises(ValueError, match="out must"):
        fq.fp8_gemm_b128(a, sa, b, sb, out=torch.zeros(6, 4, device=DEV))
    with pytest.raises(fq.Fp4qError, match="multiple of 16"):
        fq.fp8_gemm_b128(a[:, :8].contiguous(), sa, b[:, :8].contiguous(), sb)
    with pytest.raises(ValueError, match="kind"):
        fq.fp8_quantize_b128(torch.zeros(4, 4, device=DEV), 3)
    with pytest.raises(ValueError, match="nothing"):
        fq.fp8_quantize_b128(torch.zeros(4, 4, device=DEV), codes=False)
    with pytest.raises(TypeError):
        fq.fp8_quantize_b128(torch.zeros(4, 4, device=DEV, dtype=torch.float16))


def test_on_another_stream():
    """The calls run on torch's current stream, workspace included."""
    a, b = operand(100, 2048, 10, False), operand(200, 2048, 11, True)
    want = product(a, b, TILE)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = product(a, b, TILE)
    np.testing.assert_array_equal(got, want)


def linear_ref(x, w, dy):
    v = lambda t, tile: ref.value(*ref.quantize(np.ascontiguousarray(t), tile), tile)[:, :t.shape[1]]
    y, dx, dw = (v(x, False), v(w, True).T), (v(dy, False), v(w, True)), (v(dy.T, False), v(x.T, False).T)
    return [(a @ b, np.abs(a) @ np.abs(b), a.shape[1]) for a, b in (y, dx, dw)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,n,k", [(1, 3, 5), (37, 130, 70), (129, 257, 96), (300, 64, 520)])
def test_linear_and_its_gradients(t, n, k, dtype):
    rng = np.random.default_rng([12, t, n, k])
    mk = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dtype)
    x, w, dy = mk(t, k), mk(n, k), mk(t, n)
    xd, wd = x.to(DEV).requires_grad_(), w.to(DEV).requires_grad_()
    y = fq.fp8_linear(xd, wd)
    y.backward(dy.to(DEV))
    for got, (want, size, kk) in zip((y, xd.grad, wd.grad), linear_ref(x.float().numpy(), w.float().numpy(), dy.float().numpy())):
        assert got.dtype == dtype
        err = np.abs(got.detach().float().cpu().numpy() - want)
        bf16 = dtype == torch.bfloat16
        assert np.all(err <= (2.0 ** -14 * size + 2.0 ** -8 * np.abs(want) if bf16 else (kk / 128 + 8) * 2.0 ** -23 * size))


def test_linear_gradients_against_differences():
    """On values that their quantization keeps (whole numbers with 448 in every block, scales of 1) the layer is its
    product, so that differences of sum(dy y) are exact: dx and dw equal them."""
    t, n, k = 6, 5, 7
    rng = np.random.default_rng(13)
    mk = lambda *s: rng.integers(-8, 9, s).astype(np.float32)
    x, w, dy = mk(t, k), mk(n, k), mk(t, n)
    x[:, 0] = x[0, :] = 448.0
    w[0, 0] = 448.0
    dy[:, 0] = dy[0, :] = 448.0

    def loss(x, w):
        return float((fq.fp8_linear(dev(x), dev(w)).cpu().double().numpy() * dy).sum())

    xd, wd = dev(x).requires_grad_(), dev(w).requires_grad_()
    fq.fp8_linear(xd, wd).backward(dev(dy))
    for a, grad in ((x, xd.grad), (w, wd.grad)):
        for i in rng.permutation(a.size)[:12]:
            at = np.unravel_index(i, a.shape)
            if abs(a[at]) == 448.0:
                continue
            up, down = a.copy(), a.copy()
            up[at] += 1
            down[at] -= 1
            args = (lambda v: (v, w)) if a is x else (lambda v: (x, v))
            assert (loss(*args(up)) - loss(*args(down))) / 2 == float(grad[at])


def test_linear_shapes_and_what_needs_no_gradient():
    x, w = torch.randn(2, 3, 48, device=DEV), torch.randn(20, 48, device=DEV)
    assert fq.fp8_linear(x, w).shape == (2, 3, 20)
    assert fq.fp8_linear(x[0, 0], w).shape == (20,)
    assert fq.fp8_linear(x[:0], w).shape == (0, 3, 20)
    full = fq.fp8_linear(x.transpose(0, 1), w)
    assert torch.equal(full, fq.fp8_linear(x.transpose(0, 1).contiguous(), w))
    for gx, gw in ((True, False), (False, True)):
        a, b = x.clone().requires_grad_(gx), w.clone().requires_grad_(gw)
        fq.fp8_linear(a, b).sum().backward()  # an expanded gradient
        assert (a.grad is not None) == gx and (b.grad is not None) == gw
    e = torch.zeros(0, 48, device=DEV, requires_grad=True)
    wg = w.clone().requires_grad_()
    fq.fp8_linear(e, wg).sum().backward()
    assert torch.equal(wg.grad, torch.zeros_like(w))
    with pytest.raises(ValueError, match="last sizes"):
        fq.fp8_linear(x, w[:, :40])


@pytest.mark.parametrize("kind", [ROW, TILE])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_gemm_of_many_large_tiles(kind, out_dtype):
    """More 256 x 256 tiles than the chip holds at once, the last ones cut short in both sizes: sampled rows and
    columns within the bound."""
    m, n, k = 4100, 5003, 512
    a, b = operand(m, k, 14, False), operand(n, k, 15, kind == TILE)
    got = product(a, b, kind, out_dtype)
    rows = np.r_[0:5, 255:258, 2047:2050, 4095:4100]
    cols = np.r_[0:4, 2040:2060, 3500:3600:7, 3830:3850, 4340:4360, 4600:5003:13, 5000:5003]
    av, bv = ref.value(*a, False)[rows], ref.value(*b, kind == TILE)[cols]
    want, size = av @ bv.T, np.abs(av) @ np.abs(bv).T
    bar = (k / 128 + 8) * 2.0 ** -23 * size if out_dtype == torch.float32 else 2.0 ** -14 * size + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(got[np.ix_(rows, cols)] - want) <= bar)
    # Every element is written: no row or column is left as it was.
    f8 = lambda c: dev(c).view(torch.float8_e4m3fn)
    out = torch.full((m, n), float("nan"), dtype=out_dtype, device=DEV)
    fq.fp8_gemm_b128(f8(a[0]), dev(a[1]), f8(b[0]), dev(b[1]), kind, out=out)
    assert not torch.isnan(out).any()


@pytest.mark.parametrize("m,n", [(3, 24), (100, 24), (300, 520)])
def test_gemm_writes_where_rows_do_not_start_on_16_bytes(m, n):
    """An output whose rows are whole 16-byte units apart but start off them."""
    k = 256
    a, b = operand(m, k, 16, False), operand(n, k, 17, True)
    f8 = lambda c: dev(c).view(torch.float8_e4m3fn)
    flat = torch.zeros(m * n + 9, dtype=torch.bfloat16, device=DEV)
    out = flat[3:3 + m * n].view(m, n)
    fq.fp8_gemm_b128(f8(a[0]), dev(a[1]), f8(b[0]), dev(b[1]), TILE, out=out)
    assert torch.equal(out, fq.fp8_gemm_b128(f8(a[0]), dev(a[1]), f8(b[0]), dev(b[1]), TILE, out_dtype=torch.bfloat16))
    assert not flat[:3].any() and not flat[3 + m * n:].any()


@pytest.mark.parametrize("kind", [ROW, TILE])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n", [(5, 131), (40, 131), (300, 1033), (2304, 3601), (2305, 3606)])
def test_gemm_of_odd_rows_is_that_of_whole_ones(m, n, dtype, kind):
    """One K block, so that every tile size forms the same sums: C with rows that end inside 16 bytes equals the
    columns of a wider one, and nothing around it is written."""
    k, wide = 128, (n + 127) // 128 * 128
    a, b = operand(m, k, 18, False), operand(n, k, 19, kind == TILE)
    f8 = lambda c: dev(c).view(torch.float8_e4m3fn)
    more = np.zeros((wide - n, b[0].shape[1]), np.uint8)
    scales = b[1] if kind == TILE else np.concatenate([b[1], np.ones((1, wide - n), np.float32)], 1)
    want = fq.fp8_gemm_b128(f8(a[0]), dev(a[1]), f8(np.concatenate([b[0], more])), dev(scales), kind, out_dtype=dtype)
    flat = torch.zeros(m * n + 32, dtype=dtype, device=DEV)
    out = flat[16:16 + m * n].view(m, n)
    fq.fp8_gemm_b128(f8(a[0]), dev(a[1]), f8(b[0]), dev(b[1]), kind, out=out)
    assert torch.equal(out, want[:, :n])
    assert not flat[:16].any() and not flat[16 + m * n:].any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,n,k", [(5, 40, 33), (200, 300, 260), (70, 1000, 4100)])
def test_linear_is_the_calls_that_it_stands_for(t, n, k, dtype):
    rng = np.random.default_rng([18, t, n, k])
    mk = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dtype).to(DEV)
    x, w, dy = mk(t, k).requires_grad_(), mk(n, k).requires_grad_(), mk(t, n)
    y = fq.fp8_linear(x, w)
    y.backward(dy)
    xq, wq = fq.fp8_quantize_b128(x.detach(), ROW, transposed=True), fq.fp8_quantize_b128(w.detach(), TILE, transposed=True)
    dq = fq.fp8_quantize_b128(dy, ROW, transposed=True)
    assert torch.equal(y, fq.fp8_gemm_b128(xq.codes, xq.scales, wq.codes, wq.scales, TILE, dtype))
    assert torch.equal(x.grad, fq.fp8_gemm_b128(dq.codes, dq.scales, wq.codes_t, wq.scales_t, TILE, dtype))
    assert torch.equal(w.grad, fq.fp8_gemm_b128(dq.codes_t, dq.scales_t, xq.codes_t, xq.scales_t, ROW, dtype))


def test_linear_of_mixed_types():
    x = torch.randn(9, 64, device=DEV, dtype=torch.bfloat16, requires_grad=True)
    w = torch.randn(20, 64, device=DEV, requires_grad=True)
    y = fq.fp8_linear(x, w)
    y.sum().backward()
    assert y.dtype == x.grad.dtype == torch.bfloat16 and w.grad.dtype == torch.float32


def test_quantize_past_32_bits():
    """Elements and codes beyond 2^31: the last rows are those of the rows alone."""
    rows, cols = 270001, 8000
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    tail = torch.randn(257, cols, dtype=torch.bfloat16, device=DEV)
    x[-257:] = tail
    q, want = fq.fp8_quantize_b128(x), fq.fp8_quantize_b128(tail)
    assert torch.equal(q.codes[-257:].view(torch.uint8), want.codes.view(torch.uint8))
    assert torch.equal(q.scales[:, -257:], want.scales)


@pytest.mark.parametrize("m", [2, 40])
def test_gemm_past_32_bits(m):
    """B beyond 2^31 bytes, sums exact on whole numbers: the last columns are those of B's last rows alone."""
    n, k = 262400, 8320
    g = torch.Generator(device=DEV).manual_seed(3)
    small = lambda r: torch.randint(-2, 3, (r, k), generator=g, device=DEV).to(torch.float8_e4m3fn)
    a, tail = small(m), small(256)
    b = torch.zeros(n, k, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    b[-256:].view(torch.uint8).copy_(tail.view(torch.uint8))
    one = lambda *shape: torch.ones(*shape, device=DEV)
    got = fq.fp8_gemm_b128(a, one(k // 128, m), b, one(n // 128, k // 128))
    want = a.double() @ tail.double().T
    assert torch.equal(got[:, -256:].double(), want) and not got[:, :-256].any()
