"""moe_layer at sizes that take each of its kernels: gate and up by 128 rows, several
slots per expert, the router by K ranges and over each number of experts per lane.
The bars are those of the layer's other tests."""
import numpy as np
import pytest
import torch

import microscaling_fp4_quantization_amd as fq
from test_gpu_moe import DEV, FORMATS, Layer

pytestmark = pytest.mark.gpu


def workgroups(t, d, i, e, k):
    """Workgroups of gate and up by 128 rows, and how many make the layer take that form: 384, or
    224 where slots (an expert and up to 16 of its tokens) are half full."""
    slots = min(t * k, e + t * k // 16)
    return slots * -(-2 * i // 128), 224 if t * k >= 8 * slots else 384


# tokens, dim, inter, experts, top_k.  inter ends inside a workgroup's 64 rows of gate; dims that
# are and are not whole pairs of 128.
MANY = [(64, 256, 480, 40, 8), (64, 288, 1056, 8, 2), (30, 160, 672, 40, 4), (3, 512, 4128, 6, 2)]


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", MANY)
def test_gate_and_up_by_128_rows(size, dtype, fmt):
    have, need = workgroups(*size)
    assert have >= need
    m = Layer(*size, fmt, dtype, 11)
    ids, p, dp = m.routing()
    if size[0] == 64:
        assert np.bincount(ids.reshape(-1)).max() > 16  # an expert of two slots
    r = m.run()
    np.testing.assert_array_equal(r.topk_ids.cpu().numpy(), ids)
    m.check(r, ids, p, dp)


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_given_routing_by_128_rows(fmt):
    """Everyone at one expert, which fills four slots; ids that name nobody; an expert named twice."""
    t, d, i, e, k = 64, 256, 480, 40, 8
    assert workgroups(t, d, i, e, k)[0] >= 384
    m = Layer(t, d, i, e, k, fmt, torch.float32, 12)
    rng = np.random.default_rng(13)
    ids = rng.integers(-2, e + 2, (t, k)).astype(np.int32)
    ids[:, 0] = 7
    ids[5, 1:3] = 9
    ids[t - 1] = -1
    p = rng.standard_normal((t, k)).astype(np.float32)
    r = m.run(topk_ids=torch.from_numpy(ids).to(DEV), topk_weights=torch.from_numpy(p).to(DEV), out_dtype=torch.bfloat16)
    m.check(r, ids.astype(np.int64), p.astype(np.float64), np.abs(p) * 4 * 2.0 ** -23)
    assert not r.y[t - 1].any()


# The router's K ranges: (tokens, dim, experts, top_k, ranges) for 4, 8 and 32 experts per lane.
ROUTES = [(3, 2048, 60, 4, 8), (2, 2048, 100, 3, 8), (33, 1056, 128, 16, 2), (3, 544, 200, 4, 2),
          (16, 1056, 129, 16, 3), (1, 512, 300, 8, 1)]


@pytest.mark.parametrize("dtype,r_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                           (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("t,d,e,k,ranges", ROUTES)
def test_router_by_k_ranges(t, d, e, k, ranges, dtype, r_dtype):
    tiles, most = -(-e // 16) * -(-t // 16), min(8, -(-2 * d // 32 // 16))
    assert ranges == max(1, min(most, (64 if e <= 128 else 32) // tiles))
    m = Layer(t, d, 32, e, k, "mxfp4", dtype, 16, r_dtype)
    for renorm in (True, False):
        ids, p, dp = m.routing(renorm)
        r = m.run(renormalize=renorm)
        np.testing.assert_array_equal(r.topk_ids.cpu().numpy(), ids)
        assert np.all(np.abs(r.topk_weights.cpu().numpy() - p) <= dp)
    m.check(m.run(), *m.routing())


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_an_expert_past_32_bits_against_64_bits(fmt):
    """The last expert of a stack of over 2^31 bytes, within the layer's bar."""
    m = Layer(3, 2048, 2304, 1, 1, fmt, torch.bfloat16, 15)
    e = (1 << 31) // m.w13.codes.numel() + 2
    assert e <= 512

    def stack(w):
        codes = torch.zeros(e * w.codes.shape[0], w.codes.shape[1], dtype=torch.uint8, device=DEV)
        codes[-w.codes.shape[0]:] = w.codes.view(torch.uint8)
        scales = w.scales.new_zeros(e * w.scales.shape[0], w.scales.shape[1])
        scales[-w.scales.shape[0]:] = w.scales
        return fq.ExpertWeights(w.fmt, codes.view(w.codes.dtype), scales, w.g)

    m.w13, m.w2 = stack(m.w13), stack(m.w2)
    ids, wts = torch.full((3, 1), e - 1, dtype=torch.int32, device=DEV), torch.ones(3, 1, device=DEV)
    r = fq.moe_layer(m.x.to(DEV), m.w13, m.w2, e, 1, topk_ids=ids, topk_weights=wts)
    m.check(r, np.zeros((3, 1), np.int64), np.ones((3, 1)), np.zeros((3, 1)))
