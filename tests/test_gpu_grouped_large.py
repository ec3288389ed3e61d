"""The integer and grouped products past 2^31 bytes or elements, against 64 bits on some of their
rows, and grouped ones of many large tiles."""
import pytest
import torch

import microscaling_fp4_quantization_amd as fq
from test_gpu_grouped import bar, experts_of, expect, gen, i32, quantized, sizes_to_ends, value

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROW, TILE = fq.B128_ROW, fq.B128_TILE


@pytest.fixture(autouse=True)
def freed():
    yield
    torch.cuda.empty_cache()


# More tiles of 256 than CUs, most groups ending inside one; a stacked matrix's experts may start
# inside a block of scales.
@pytest.mark.parametrize("form", ["experts", "stacked", "gathered"])
@pytest.mark.parametrize("sizes,n,k", [([4100, 200], 4300, 2048), ([4000, 3000, 100, 2200], 2200, 2064), ([14500] + [0] * 9 + [30], 2304, 2048),
                                       ([90, 6000, 255, 5700], 2000, 1920), ([17409], 1800, 2048)])
def test_many_large_tiles(sizes, n, k, form):
    g = gen(n)
    e, ends = len(sizes), sizes_to_ends(sizes)
    rows = ends[-1] + 1
    w = torch.randn(e, n, k, generator=g, device=DEV)
    if form == "stacked":
        q = fq.fp8_quantize_b128(w.view(e * n, k), TILE)
        codes, scales = q.codes, q.scales
        wv = value(codes, scales, TILE).view(e, n, -1)
    else:
        codes, scales = experts_of(w)
        wv = torch.stack([value(c, s, TILE) for c, s in zip(codes, scales)])
    qa = fq.fp8_quantize_b128(torch.randn(1000 if form == "gathered" else rows, k, generator=g, device=DEV))
    tokens = torch.randint(0, 1000, (rows,), generator=g, device=DEV, dtype=torch.int32) if form == "gathered" else None
    out = torch.full((rows, n), 77.0, dtype=torch.bfloat16, device=DEV)
    fq.fp8_grouped_gemm_b128(qa.codes, qa.scales, codes, scales, i32(ends), tokens=tokens, out=out)
    want, size = expect(value(qa.codes, qa.scales, ROW), wv, ends, tokens, rows)
    assert bool((out[-1] == 77.0).all())
    assert bool(((out.double() - want).abs() <= bar(want, size, k, torch.bfloat16))[:-1].all())


def int8_rows(rows, cols, seed):
    return torch.randint(-127, 128, (rows, cols), generator=gen(seed), device=DEV, dtype=torch.int8)


def test_int8_operand_past_2_31_bytes():
    m, n, k = 70000, 40, 32768
    a, b = int8_rows(m, k, 1), int8_rows(n, k, 2)
    sa, sb = torch.rand(m, device=DEV) + 0.5, torch.rand(n, device=DEV) + 0.5
    c = fq.int8_gemm(a, sa, b, sb)
    for at in (0, 65535, 65536, m - 300):
        acc = a[at:at + 300].double() @ b.double().t()
        assert torch.equal(c[at:at + 300], (acc.float().double() * (sa[at:at + 300, None] * sb).double()).float())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_int8_output_past_2_31_bytes(dtype):
    m, n, k = 300000, 4100, 128
    a, b = int8_rows(m, k, 3), int8_rows(n, k, 4)
    sa, sb = torch.rand(m, device=DEV) + 0.5, torch.rand(n, device=DEV) + 0.5
    c = fq.int8_gemm(a, sa, b, sb, out_dtype=dtype)
    for at in (0, 130900, 261800, m - 500):
        acc = a[at:at + 500].double() @ b.double().t()
        assert torch.equal(c[at:at + 500], (acc.float().double() * (sa[at:at + 500, None] * sb).double()).float().to(dtype))


def test_int8_quantize_past_2_31_elements():
    x = torch.empty(70000, 32768, dtype=torch.bfloat16, device=DEV)
    for at in range(0, 70000, 10000):
        x[at:at + 10000] = torch.randn(10000, 32768, generator=gen(at), device=DEV).bfloat16()
    q = fq.int8_quantize_rows(x)
    for at in (0, 65530, 69990):
        some = fq.int8_quantize_rows(x[at:at + 10].contiguous())
        assert torch.equal(q.codes[at:at + 10], some.codes) and torch.equal(q.scales[at:at + 10], some.scales)


@pytest.mark.parametrize("rows", [30, 1200])
def test_grouped_weights_past_2_31_bytes(rows):
    e, n, k = 40, 2048, 32768
    codes = torch.empty(e, n, k, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty(e, n // 128, k // 128, device=DEV)
    for i in range(e):
        q = fq.fp8_quantize_b128(torch.randn(n, k, generator=gen(i), device=DEV), TILE)
        codes[i], scales[i] = q.codes, q.scales
    qa = fq.fp8_quantize_b128(torch.randn(rows, k, generator=gen(99), device=DEV))
    sizes = [0] * e
    sizes[0], sizes[31], sizes[33], sizes[39] = rows // 3, rows // 3, 1, rows - 2 * (rows // 3) - 1
    ends = sizes_to_ends(sizes)
    c = fq.fp8_grouped_gemm_b128(qa.codes, qa.scales, codes, scales, i32(ends))
    av = value(qa.codes, qa.scales, ROW)
    for i in (0, 31, 33, 39):
        wv = value(codes[i], scales[i], TILE)
        x = av[ends[i]:ends[i + 1]]
        want, size = x @ wv.t().contiguous(), x.abs() @ wv.abs().t().contiguous()
        assert bool(((c[ends[i]:ends[i + 1]].double() - want).abs() <= bar(want, size, k, torch.float32)).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_grouped_output_past_2_31_bytes(dtype):
    rows, n, k = 300000, 4104, 128
    codes, scales = experts_of(torch.randn(3, n, k, generator=gen(5), device=DEV))
    qa = fq.fp8_quantize_b128(torch.randn(rows, k, generator=gen(6), device=DEV))
    ends = [0, 100001, 100001, rows]
    c = fq.fp8_grouped_gemm_b128(qa.codes, qa.scales, codes, scales, i32(ends), out_dtype=dtype)
    for e, at in ((0, 0), (0, 99700), (2, 100001), (2, 200000), (2, rows - 300)):
        x = value(qa.codes[at:at + 300], qa.scales[:, at:at + 300], ROW)
        wv = value(codes[e], scales[e], TILE)
        want, size = x @ wv.t().contiguous(), x.abs() @ wv.abs().t().contiguous()
        assert bool(((c[at:at + 300].double() - want).abs() <= bar(want, size, k, dtype)).all())


def test_grouped_linear_of_weights_past_2_31_elements():
    rows, e, n, k = 300, 66, 8200, 4096
    w = torch.empty(e, n, k, dtype=torch.bfloat16, device=DEV)
    for i in range(e):
        w[i] = torch.randn(n, k, generator=gen(i), device=DEV).bfloat16()
    w.requires_grad_()
    x = torch.randn(rows, k, generator=gen(100), device=DEV).bfloat16().requires_grad_()
    dy = torch.randn(rows, n, generator=gen(101), device=DEV).bfloat16()
    sizes = [0] * e
    sizes[0], sizes[63], sizes[64], sizes[65] = 100, 50, 20, 130
    ends = sizes_to_ends(sizes)
    y = fq.fp8_grouped_linear(x, w, i32(ends))
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    for i in (0, 63, 64, 65):
        at = slice(ends[i], ends[i + 1])
        xe, dye, wq = x.detach()[at], dy[at], quantized(w.detach()[i], TILE)
        for got, a, b, terms in ((y.detach()[at], quantized(xe), wq, k), (dx[at], quantized(dye), wq.t(), n), (dw[i], quantized(dye.t()), quantized(xe.t()), 256)):
            want, size = a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()
            assert bool(((got.double() - want).abs() <= bar(want, size, terms, torch.bfloat16)).all())
    assert bool((dw[1] == 0).all()) and bool((dw[62] == 0).all())
