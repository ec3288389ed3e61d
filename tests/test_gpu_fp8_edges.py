"""The 8-bit operators where nothing, or nothing finite, comes in."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
import microscaling_fp4_quantization_amd as fq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROW, TILE = fq.B128_ROW, fq.B128_TILE


@pytest.mark.parametrize("shape", [(2, 3, 0), (0, 3, 0), (3, 0), (0,), (2, 0, 16), (0, 2, 16)])
def test_linear_of_empty_inputs(shape):
    """Any number of dimensions, no features or no tokens: zeros of the right shapes."""
    x = torch.zeros(shape, device=DEV, requires_grad=True)
    w = torch.zeros(5, shape[-1], device=DEV, requires_grad=True)
    y = fq.fp8_linear(x, w)
    assert y.shape == (*shape[:-1], 5) and not y.any()
    y.backward(torch.ones_like(y))
    assert x.grad.shape == shape and w.grad.shape == w.shape and not x.grad.any() and not w.grad.any()
    assert fq.fp8_linear(x, w[:0]).shape == (*shape[:-1], 0)


def same_but_nan(got, want):
    """Equal codes, with either sign of NaN."""
    nan = (want & 0x7F) == 0x7F
    np.testing.assert_array_equal((got & 0x7F) == 0x7F, nan)
    np.testing.assert_array_equal(got[~nan], want[~nan])


def reference(x, tile):
    """fp8_ref's codes and scales with each NaN taken as 0 first, then a NaN code; blocks of an infinity by hand."""
    nan, inf = np.isnan(x), np.isinf(x)
    codes, scales = ref.quantize(np.where(nan | inf, 0, x).astype(np.float32), tile)
    step = 128 if tile else 1
    s = scales if tile else scales.T
    for r, c in np.argwhere(inf):
        block = (slice(r // step * step, r // step * step + step), slice(c // 128 * 128, min(x.shape[1], c // 128 * 128 + 128)))
        codes[block] = np.where(inf[block], 0x7F, np.where(np.signbit(x[block]), 0x80, 0))
        s[r // step, c // 128] = np.inf
    codes[:, :x.shape[1]][nan] = 0x7F
    return codes, scales


@pytest.mark.parametrize("kind", [ROW, TILE])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_keeps_what_is_not_finite_in_its_block(dtype, kind):
    rng = np.random.default_rng(21)
    t = torch.from_numpy(rng.standard_normal((300, 290)).astype(np.float32)).to(dtype)
    for r, c, v in ((3, 5, "nan"), (3, 200, "-nan"), (140, 7, "inf"), (299, 289, "-inf"), (260, 131, "nan"), (9, 250, "nan")):
        t[r, c] = float(v)
    t[200] = float("nan")
    x = t.float().numpy()
    q = fq.fp8_quantize_b128(t.to(DEV), kind, transposed=True)
    for codes, scales, src in ((q.codes, q.scales, x), (q.codes_t, q.scales_t, x.T)):
        c, s = reference(src, kind == TILE)
        np.testing.assert_array_equal(scales.cpu().numpy(), s)
        same_but_nan(codes.view(torch.uint8).cpu().numpy(), c)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_linear_shows_what_is_not_finite(value):
    """One such element of x: its row of y and its column of dw are NaN; of dy: its row of dx and of dw."""
    x, w, dy = torch.randn(40, 96, device=DEV), torch.randn(56, 96, device=DEV), torch.randn(40, 56, device=DEV)
    for at in ("x", "dy"):
        a, g = x.clone(), dy.clone()
        (a if at == "x" else g)[7, 11] = value
        a, b = a.requires_grad_(), w.clone().requires_grad_()
        y = fq.fp8_linear(a, b)
        y.backward(g)
        rows = torch.arange(40, device=DEV) == 7
        assert torch.equal(torch.isnan(y).all(1), rows & (at == "x"))
        assert torch.equal(torch.isnan(y).any(1), rows & (at == "x"))
        assert torch.equal(torch.isnan(a.grad).any(1), rows & (at == "dy"))
        hit = torch.zeros(56, 96, dtype=torch.bool, device=DEV)
        if at == "x":
            hit[:, 11] = True
        else:
            hit[11] = True
        assert torch.equal(torch.isnan(b.grad), hit)


def test_a_backward_pass_through_calls_without_a_gradient_raises():
    a, b = fq.fp8_quantize_b128(torch.randn(20, 64, device=DEV)), fq.fp8_quantize_b128(torch.randn(30, 64, device=DEV), TILE)
    want = fq.fp8_gemm_b128(a.codes, a.scales, b.codes, b.scales)
    s = b.scales.clone().requires_grad_()
    for out in (None, torch.empty_like(want)):
        y = fq.fp8_gemm_b128(a.codes, a.scales, b.codes, s, out=out)
        assert torch.equal(y, want)
        assert out is None or (y.data_ptr() == out.data_ptr() and not out.requires_grad)
        with pytest.raises(NotImplementedError, match="fp8_gemm_b128"):
            y.sum().backward()
    with torch.no_grad():
        assert not fq.fp8_gemm_b128(a.codes, a.scales, b.codes, s).requires_grad

    e, d, i, k, t = 4, 64, 32, 2, 3
    quant = lambda r, c: fq.fp8_quantize_b128(torch.randn(r, c, device=DEV), TILE)
    w13, w2 = (fq.ExpertWeights(fq.FMT_E4M3_B128, q.codes, q.scales) for q in (quant(e * 2 * i, d), quant(e * d, i)))
    x, wr = torch.randn(t, d, device=DEV), torch.randn(e, d, device=DEV)
    want = fq.moe_layer(x, w13, w2, e, k, router=wr)
    assert not want.y.requires_grad
    for xg, rg in ((True, False), (False, True)):
        r = fq.moe_layer(x.clone().requires_grad_(xg), w13, w2, e, k, router=wr.clone().requires_grad_(rg))
        assert torch.equal(r.y, want.y) and torch.equal(r.topk_weights, want.topk_weights)
        for v in (r.y, r.topk_weights):
            with pytest.raises(NotImplementedError, match="moe_layer"):
                v.sum().backward(retain_graph=True)
    w = want.topk_weights.clone().requires_grad_()
    r = fq.moe_layer(x, w13, w2, e, k, topk_ids=want.topk_ids, topk_weights=w)
    assert torch.equal(r.y, want.y)
    with pytest.raises(NotImplementedError, match="moe_layer"):
        r.y.sum().backward()
    with torch.no_grad():
        assert not fq.moe_layer(x.clone().requires_grad_(), w13, w2, e, k, router=wr).y.requires_grad
