"""Rows that no group owns: before the first group, behind the last, and slots of no expert.

Memory that a call gets is filled with NaN first, so that an output that is not written shows.
Bounds as in test_gpu_grouped.py."""
import pytest
import torch

import microscaling_fp4_quantization_amd as fq
from test_gpu_grouped import TYPES, bar, gen, i32, linear_expect

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
    ends = [first]
    for m in sizes:
        ends.append(ends[-1] + m)
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
