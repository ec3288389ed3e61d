"""The shapes of the kernel tests take the kernels that they are there for (on the CPU)."""
import random

import pytest

import tile_choice
from test_abi import L  # noqa: F401  (the loaded library, built if it is missing)
from test_gpu_grouped_kernels import PRODUCTS, STACKED, STEPS
from test_gpu_int8_kernels import LARGE, RANGES


@pytest.mark.parametrize("shape,want", [*LARGE.items(), *RANGES.items()])
def test_int8(shape, want):
    assert tile_choice.int8(*shape) == want


@pytest.mark.parametrize("shape,bf16,f32", STEPS)
def test_grouped_steps(shape, bf16, f32):
    sizes, n, k = shape
    rows, e = sum(sizes) + 5, len(sizes)
    for wide, want in ((False, bf16), (True, f32)):
        got = (tile_choice.grouped(rows, e + 1, n, k, wide), tile_choice.grouped(rows, e + 1, k, n, wide), tile_choice.outer(rows, e, n, k, wide))
        assert got == want


@pytest.mark.parametrize("shape,bf16,f32", PRODUCTS + STACKED)
def test_grouped_products(shape, bf16, f32):
    sizes, n, k = shape
    assert (tile_choice.grouped(sum(sizes) + 3, len(sizes), n, k, False), tile_choice.grouped(sum(sizes) + 3, len(sizes), n, k, True)) == (bf16, f32)


def test_int8_formulas_are_the_librarys(L):
    """Its workspace holds the K ranges' sums: as many ranges as the formulas here give."""
    rng = random.Random(7)
    size = lambda lo, hi: int(lo * (hi / lo) ** rng.random())
    shapes = [*LARGE, *RANGES] + [(size(17, 9000), size(1, 9000), 16 * size(1, 8191)) for _ in range(3000)]
    ranges = set()
    for m, n, k in shapes:
        tile, sp, _ = tile_choice.int8(m, n, k)
        ranges.add((tile, sp))
        assert L.int8_gemm_workspace_bytes(m, n, k) == (4 * sp * m * n if sp > 1 else 0), (m, n, k)
    assert len(ranges) > 12
