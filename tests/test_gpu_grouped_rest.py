"""Rows that no group owns: before the first group, behind the last, and slots of no expert.

Memory that a call gets is filled with NaN first, so that an output that is not written shows.
Bounds as in test_gpu_grouped.py."""
import pytest
import torch

import microscaling_fp4_quantization_amd as fq
from test_gpu_grouped import TYPES, bar, experts_of, gen, i32, linear_expect, sizes_to_ends

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dirty(*shapes, dtype):
    """Leaves NaN in the free memory that tensors of these shapes are likely to get."""
    held = [torch.full(s, float("nan"), dtype=dtype, device=DEV) for s in shapes for _ in range(3)]
    torch.cuda.synchronize()
    del held


# Rows before the first group, sizes of the groups, rows behind the last, N, K: the pass over the
# weights, tiles of 64, 128 and 256, and as many tiles as rows of no group can take.
RUNS = [(3, [2, 0, 5], 4, 40, 72), (1, [1] * 9, 1, 130, 256), (30, [0, 3], 0, 16, 16), (70, [0, 65, 130], 33, 200, 136), (1, [65, 1, 129], 1, 96, 128),
        (200, [0, 0], 100, 64, 64), (1000, [900, 0, 1700], 500, 1024, 512), (1, [3000, 0, 1700, 2500, 5001, 1100], 1, 2048, 2048)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("first,sizes,last,n,k", RUNS)
def test_linear_of_a_run_of_experts(first, sizes, last, n, k, dtype):
    """w and offsets of some of a batch's experts: the other experts' rows are zeros in y and dx,
    whatever x and dy hold there, and no part of dw."""
    g = gen(n + k + first)
    ends = sizes_to_ends([first] + sizes)[1:]
    rows = ends[-1] + last
    x = torch.randn(rows, k, generator=g, device=DEV).to(dtype)
    dy = torch.randn(rows, n, generator=g, device=DEV).to(dtype)
    x[:first], x[ends[-1]:], dy[:first], dy[ends[-1]:] = float("nan"), float("inf"), float("inf"), float("nan")
    w = (torch.randn(len(sizes), n, k, generator=g, device=DEV) * 0.1).to(dtype).requires_grad_()
    x.requires_grad_()
    whole = i32([0] + ends + [rows])
    dirty((rows, n), (rows, k), dtype=dtype)
    y = fq.fp8_grouped_linear(x, w, whole[1:-1])
    dirty((rows, k), tuple(w.shape), dtype=dtype)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    want = linear_expect(x.detach(), w.detach(), dy, ends)
    for name, got, terms in (("y", y.detach(), k), ("dx", dx, n), ("dw", dw, max(sizes))):
        v, size = want[name]
        assert bool(((got.double() - v).abs() <= bar(v, size, terms, got.dtype)).all()), name
    for t in (y, dx):
        assert bool((t[:first] == 0).all()) and bool((t[ends[-1]:] == 0).all())


@pytest.mark.parametrize("n,k", [(40, 72), (264, 136)])
def test_linear_of_wrong_offsets_is_finite(n, k):
    """Offsets out of order or outside the rows: what comes out is products or zeros of finite rows."""
    g = gen(n)
    rows = 600
    x = torch.randn(rows, k, generator=g, device=DEV, requires_grad=True)
    w = torch.randn(4, n, k, generator=g, device=DEV, requires_grad=True)
    dy = torch.randn(rows, n, generator=g, device=DEV)
    for ends in ([300, 200, 100, 0, 0], [-7, -7, -7, -7, -7], [900, 900, 900, 900, 900], [600, 0, 0, 0, 600], [5, 400, 400, 9000, 9000]):
        dirty((rows, n), (rows, k), dtype=torch.float32)
        y = fq.fp8_grouped_linear(x, w, i32(ends))
        dx, dw = torch.autograd.grad(y, (x, w), dy)
        assert all(bool(t.isfinite().all()) for t in (y, dx, dw)), ends
        if max(ends) <= 0 or min(ends) >= rows:
            assert not any(bool(t.any()) for t in (y, dx, dw))


# ---------------------------------------------------------------------------
# The product, and slots of no expert


# As RUNS, and [8] * 16, where one group more would take another kernel.
PRODUCTS = RUNS + [(0, [8] * 16, 3, 256, 1024), (2, [8] * 16, 1, 256, 1024), (0, [70, 0, 65], 0, 200, 272)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("form", ["experts", "stacked", "gathered"])
@pytest.mark.parametrize("first,sizes,last,n,k", PRODUCTS)
def test_product_clears_rows_of_no_group(first, sizes, last, n, k, form, dtype):
    """clear_rest: zeros before the first group and behind the last, the same bits in the groups;
    A's rows, gathered or not, do not come into it where no group is."""
    g = gen(n + k + first)
    ends = sizes_to_ends([first] + sizes)
    rows, e = ends[-1] + last, len(sizes)
    w = torch.randn(e, n, k, generator=g, device=DEV)
    if form == "stacked":
        q = fq.fp8_quantize_b128(w.view(e * n, k), fq.B128_TILE)
        codes, scales = q.codes, q.scales
    else:
        codes, scales = experts_of(w)
    a_rows = rows // 2 + 1 if form == "gathered" else rows
    qa = fq.fp8_quantize_b128(torch.randn(a_rows, k, generator=g, device=DEV))
    tokens = torch.randint(0, a_rows, (rows,), generator=g, device=DEV, dtype=torch.int32) if form == "gathered" else None
    if tokens is None:
        qa.codes.view(torch.uint8)[:first], qa.codes.view(torch.uint8)[ends[-1]:] = 0x7F, 0x7F  # NaN
    offsets = i32(ends[1:])
    buf = torch.full((rows + 2, n), float("nan"), dtype=dtype, device=DEV)
    out = fq.fp8_grouped_gemm_b128(qa.codes, qa.scales, codes, scales, offsets, tokens=tokens, out=buf[1:-1], clear_rest=True)
    plain = fq.fp8_grouped_gemm_b128(qa.codes, qa.scales, codes, scales, offsets, tokens=tokens, out=torch.full_like(out, 5.0))
    assert torch.equal(out[first:ends[-1]], plain[first:ends[-1]]) and bool(out.isfinite().all())
    for rest in (slice(0, first), slice(ends[-1], rows)):
        assert bool((out[rest] == 0).all()) and bool((plain[rest] == 5.0).all())
    assert bool(buf[0].isnan().all()) and bool(buf[-1].isnan().all())


@pytest.mark.parametrize("dropped", [0.0, 0.2, 1.0])
@pytest.mark.parametrize("tokens", [1, 9, 300])
def test_a_prompt_with_dropped_slots(tokens, dropped):
    """Slots of no expert add nothing to the weighted sum, with a weight of 0 or any other."""
    g = gen(tokens)
    dim, inter, experts, top_k = 128, 64, 6, 2
    w13, w2 = (fq.fp8_quantize_b128(torch.randn(experts * r, c, generator=g, device=DEV) * c ** -0.5, fq.B128_TILE)
               for r, c in ((2 * inter, dim), (dim, inter)))
    h = torch.randn(tokens, dim, generator=g, device=DEV)
    weights, ids = torch.softmax(torch.randn(tokens, experts, generator=g, device=DEV), 1).topk(top_k)
    kept = torch.rand(ids.shape, generator=g, device=DEV) >= dropped

    def layer(ids, weights):
        o = fq.expert_order(ids, experts)
        q = fq.fp8_quantize_b128(h)
        dirty((tokens * top_k, 2 * inter), (tokens * top_k, dim), dtype=torch.float32)
        gate, up = fq.fp8_grouped_gemm_b128(q.codes, q.scales, w13.codes, w13.scales, o.offsets, tokens=o.tokens).chunk(2, 1)
        a = fq.fp8_quantize_b128((torch.nn.functional.silu(gate) * up).contiguous())
        dirty((tokens * top_k, 2 * inter), (tokens * top_k, dim), dtype=torch.float32)
        down = fq.fp8_grouped_gemm_b128(a.codes, a.scales, w2.codes, w2.scales, o.offsets, clear_rest=True)
        return (down[o.position.long()] * weights[..., None]).sum(1)

    whole, some = layer(ids, weights * kept), torch.where(kept, ids, -1)
    assert torch.equal(layer(some, weights * kept), whole) and torch.equal(layer(some, weights), whole)
