"""Workspaces that a caller gives to the grouped and the integer operators: taken where a kernel can
write them, refused before any launch elsewhere (the host's memory, another type, one byte repeated)."""
import pytest
import torch

import microscaling_fp4_quantization_amd as fq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def cases():
    x = torch.randn(100, 8192, device=DEV)
    w = fq.int8_quantize_rows(torch.randn(256, 8192, device=DEV))
    a = fq.int8_quantize_rows(x)
    ids = torch.randint(0, 128, (16384, 8), device=DEV, dtype=torch.int32)
    lib = fq.lib()
    return {
        "expert_order": (lib.expert_order_workspace_bytes(16384, 8, 128), lambda ws: fq.expert_order(ids, 128, ws=ws).order),
        "int8_gemm": (lib.int8_gemm_workspace_bytes(100, 256, 8192), lambda ws: fq.int8_gemm(a.codes, a.scales, w.codes, w.scales, ws=ws)),
        "int8_linear": (lib.int8_linear_workspace_bytes(100, 8192, 256), lambda ws: fq.int8_linear(x, w, ws=ws)),
    }


@pytest.mark.parametrize("name", ["expert_order", "int8_gemm", "int8_linear"])
def test_given_workspace(name):
    need, call = cases()[name]
    assert need > 0
    want = call(None)
    buf = torch.full((need + 512,), 7, dtype=torch.uint8, device=DEV)
    assert torch.equal(call(buf[256:256 + need]), want)
    assert bool((buf[:256] == 7).all()) and bool((buf[256 + need:] == 7).all())
    for bad in (torch.empty(need, dtype=torch.uint8), torch.empty(need, dtype=torch.uint8, pin_memory=True),
                torch.empty(need, dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.uint8, device=DEV).expand(need),
                torch.empty(2 * need, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError, match="ws must be contiguous uint8 on cuda:0"):
            call(bad)
    with pytest.raises(fq.Fp4qError, match="workspace"):
        call(buf[:need - 1])
