"""fp8_grouped_gemm_b128_cleared refuses what fp8_grouped_gemm_b128 does, and expert_order what the
library cannot be told, before any launch."""
import pytest
import torch

import microscaling_fp4_quantization_amd as fq
from test_abi import L, err  # noqa: F401  (the loaded library, built if it is missing)

OK, ARG, SHAPE, ALIGN = 0, 1, 2, 3
A, B, C, D, E, F = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000  # aligned addresses, never dereferenced


def test_validation(L):
    def gemm(a=A, sa=B, ar=40, b=C, sb=D, st=0, off=E, e=4, tok=None, r=40, n=96, k=64, c=F, ct=0):
        return L.fp8_grouped_gemm_b128_cleared(a, sa, ar, b, sb, st, off, e, tok, r, n, k, c, ct, None)

    assert gemm(ct=2) == ARG and err(L).startswith("fp8_grouped_gemm_b128_cleared")
    assert gemm(e=0) == SHAPE and gemm(e=513) == SHAPE and gemm(k=24) == SHAPE and gemm(n=1 << 22) == SHAPE
    assert gemm(ar=39) == SHAPE and gemm(tok=A, ar=1 << 26, k=32) == SHAPE
    assert gemm(r=(1 << 28) + 1, ar=(1 << 28) + 1) == SHAPE and "2^28" in err(L)
    for missing in ("a", "sa", "b", "sb", "off", "c"):
        assert gemm(**{missing: None}) == ARG, missing
    assert gemm(a=A + 8) == ALIGN and gemm(c=F + 1) == ALIGN and gemm(tok=A + 2) == ALIGN
    assert gemm(r=0, ar=0, a=None, sa=None, b=None, sb=None, off=None, c=None) == OK
    assert gemm(n=0, a=None, sa=None, b=None, sb=None, off=None, c=None) == OK


def test_numbers_that_32_bits_do_not_hold():
    """The library takes them in 32 bits, where 2^32 + 4 experts are 4."""
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for experts in (1 << 31, (1 << 32) + 4):
        with pytest.raises(ValueError, match="below 2\\^31"):
            fq.expert_order(ids, experts)
    with pytest.raises(ValueError, match="below 2\\^31"):
        fq.expert_order(torch.zeros(1, 1, dtype=torch.int32).expand(1, (1 << 32) + 8), 8)
