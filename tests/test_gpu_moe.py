"""moe_layer against its definition in 64 bits.

The bar of each element of y follows the arithmetic (u = 2^-23, a binary32 rounding
with a factor 2 of headroom; sums run over K in steps of 32 and end in up to 24
partial sums):
  logits   dl = (dim/32 + 24) u |x| |Wr|^T, so dp <= 2 dl p + 8 u p
  g, up    dg = (dim/32 + 24) u |G| |x|, and du alike
  h        |silu'| <= 1.1: dh = 1.1 dg |up| + |silu(g)| du + 8 u |h|, and the
           rounding of h to two bf16 parts (2^-16 |h|; three, under u, for a
           binary32 y)
  y        dy = sum p |D| dh + (inter/32 + 24 + top_k) u S + sum dp |D| |h| with
           S = sum p |D| |h|; a bf16 y adds 2^-8 |y|.
Inputs lean towards chosen experts, so that no two logits that decide are as near as dl.
"""
import numpy as np
import pytest
import torch

import fp8_ref
import oracle
import microscaling_fp4_quantization_amd as fq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FORMATS = {"mxfp4": fq.FMT_MXFP4, "nvfp4": fq.FMT_UE4M3, "fp8": fq.FMT_E4M3_B128}
U = 2.0 ** -23


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def stacked(w, fmt, g_per=0):
    """(ExpertWeights on the device, values in 64 bits) of a stacked matrix; g_per: rows per expert, for a g of each."""
    rows, k = w.shape
    if fmt == "fp8":
        c, s = fp8_ref.quantize(w, True)
        return fq.ExpertWeights(FORMATS[fmt], dev(c).view(torch.float8_e4m3fn), dev(s)), fp8_ref.value(c, s, True)
    if fmt == "mxfp4":
        q = oracle.quantize(w, oracle.FMT_MXFP4, 32)
        v = oracle.dequantize(q["codes"], q["scales"], oracle.FMT_MXFP4, 32, 1.0, rows, k)
        return fq.ExpertWeights(FORMATS[fmt], dev(q["codes"]), dev(q["scales"])), v.astype(np.float64)
    parts = [w[i:i + g_per] for i in range(0, rows, g_per)] if g_per else [w]
    codes, scales, gs, vals = [], [], [], []
    for part in parts:
        q = oracle.quantize(part, oracle.FMT_UE4M3, 16, gmode=oracle.GMODE_DYNAMIC)
        v = oracle.dequantize(q["codes"], q["scales"], oracle.FMT_UE4M3, 16, 1.0, part.shape[0], k)
        codes.append(q["codes"]), scales.append(q["scales"]), gs.append(q["g"])
        vals.append(v.astype(np.float64) * float(q["g"]))
    return (fq.ExpertWeights(FORMATS[fmt], dev(np.concatenate(codes)), dev(np.concatenate(scales)),
                             dev(np.array(gs, np.float32).reshape(-1))), np.concatenate(vals))


class Layer:
    def __init__(self, t, d, i, e, k, fmt, dtype=torch.bfloat16, seed=0, r_dtype=None, g_per=False):
        rng = np.random.default_rng([seed, t, d, i, e, k])
        self.size = t, d, i, e, k
        mk = lambda r, c: (rng.standard_normal((r, c)) * c ** -0.5).astype(np.float32)
        self.w13, self.v13 = stacked(mk(e * 2 * i, d), fmt, 2 * i if g_per else 0)
        self.w2, self.v2 = stacked(mk(e * d, i), fmt, d if g_per else 0)
        self.wr = torch.from_numpy(mk(e, d)).to(r_dtype or dtype)
        wr = self.wr.double().numpy()
        x = rng.standard_normal((t, d))
        for n in range(t):
            pick = rng.permutation(e)[:k]
            x[n] += ((4 + 0.9 * np.arange(k))[:, None] * wr[pick]).sum(0) / (wr[pick] ** 2).sum(1).mean()
        self.x = torch.from_numpy(x.astype(np.float32)).to(dtype)

    def run(self, **kw):
        t, d, i, e, k = self.size
        args = dict(router=self.wr.to(DEV)) if "topk_ids" not in kw else {}
        return fq.moe_layer(self.x.to(DEV), self.w13, self.w2, e, k, **args, **kw)

    def routing(self, renorm=True):
        t, d, i, e, k = self.size
        x, wr = self.x.double().numpy(), self.wr.double().numpy()
        l = x @ wr.T
        ids = np.argsort(-l, axis=1, kind="stable")[:, :k]
        ex = np.exp(l - l.max(1, keepdims=True))
        p = np.take_along_axis(ex, ids, 1)
        p /= p.sum(1, keepdims=True) if renorm else ex.sum(1, keepdims=True)
        dl = (d / 32 + 24) * U * (np.abs(x) @ np.abs(wr).T).max(1, keepdims=True)
        best = -np.sort(-l, axis=1)[:, :k + 1]
        assert np.all(best[:, :-1] - best[:, 1:] > 2 * dl), "inputs do not decide the routing"
        return ids, p, 2 * dl * p + 8 * U * p

    def reference(self, ids, p, dp, y32):
        t, d, i, e, k = self.size
        x = self.x.double().numpy()
        y, dy = np.zeros((t, d)), np.zeros((t, d))
        for n in range(t):
            size = np.zeros(d)
            for j in range(ids.shape[1]):
                ex = ids[n, j]
                if ex < 0 or ex >= e:
                    continue
                g, u = np.split(self.v13[ex * 2 * i:(ex + 1) * 2 * i] @ x[n], 2)
                sg, su = np.split((d / 32 + 24) * U * (np.abs(self.v13[ex * 2 * i:(ex + 1) * 2 * i]) @ np.abs(x[n])), 2)
                silu = g / (1 + np.exp(-g))
                h = silu * u
                dh = 1.1 * sg * np.abs(u) + np.abs(silu) * su + (8 * U + (U if y32 else 2.0 ** -16)) * np.abs(h)
                dn = self.v2[ex * d:(ex + 1) * d]
                y[n] += p[n, j] * (dn @ h)
                size += abs(p[n, j]) * (np.abs(dn) @ np.abs(h))
                dy[n] += abs(p[n, j]) * (np.abs(dn) @ dh) + dp[n, j] * (np.abs(dn) @ np.abs(h))
            dy[n] += (i / 32 + 24 + k) * U * size
        return y, dy

    def check(self, r, ids, p, dp):
        y32 = r.y.dtype == torch.float32
        y, dy = self.reference(ids, p, dp, y32)
        bar = dy + (0 if y32 else 2.0 ** -8 * np.abs(y))
        err = np.abs(r.y.double().cpu().numpy() - y)
        assert np.all(err <= bar), f"{np.max(err / np.maximum(bar, 1e-300))} of the bar"


# Tokens: one, inside a fragment, two, three and four fragments; sizes that end inside a
# step of 128 and inside a wave's share; experts below and over a wave's 64 lanes.
SIZES = [(1, 32, 32, 1, 1), (1, 256, 128, 8, 2), (3, 96, 160, 5, 5), (7, 896, 480, 12, 3), (16, 160, 64, 20, 4),
         (17, 128, 96, 70, 6), (33, 256, 64, 3, 2), (64, 192, 96, 9, 3), (64, 64, 32, 130, 8), (2, 4128, 32, 6, 2),
         (5, 64, 2080, 4, 2)]


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", SIZES)
def test_layer_is_the_definition(size, dtype, fmt):
    m = Layer(*size, fmt, dtype)
    ids, p, dp = m.routing()
    r = m.run()
    np.testing.assert_array_equal(r.topk_ids.cpu().numpy(), ids)
    assert np.all(np.abs(r.topk_weights.cpu().numpy() - p) <= dp)
    m.check(r, ids, p, dp)


@pytest.mark.parametrize("x_dtype,r_dtype,out", [(torch.bfloat16, torch.float32, torch.float32),
                                                 (torch.float32, torch.bfloat16, torch.bfloat16),
                                                 (torch.bfloat16, torch.bfloat16, torch.float32)])
def test_mixed_types_and_weights_over_all_experts(x_dtype, r_dtype, out):
    m = Layer(9, 224, 96, 11, 3, "mxfp4", x_dtype, 1, r_dtype)
    ids, p, dp = m.routing(renorm=False)
    r = m.run(renormalize=False, out_dtype=out)
    assert r.y.dtype == out
    np.testing.assert_array_equal(r.topk_ids.cpu().numpy(), ids)
    assert np.all(np.abs(r.topk_weights.cpu().numpy() - p) <= dp)
    m.check(r, ids, p, dp)


def test_one_g_per_expert():
    m = Layer(6, 128, 64, 5, 2, "nvfp4", torch.float32, 2, g_per=True)
    assert m.w13.g.numel() == 5
    ids, p, dp = m.routing()
    m.check(m.run(), ids, p, dp)


def test_equal_logits_go_to_the_lowest_index():
    t, e, k = 3, 100, 5
    m = Layer(t, 64, 32, e, k, "mxfp4", torch.bfloat16, 3)
    m.wr = m.wr[:1].expand(e, -1).contiguous()
    np.testing.assert_array_equal(m.run().topk_ids.cpu().numpy(), np.tile(np.arange(k), (t, 1)))
    m.wr = torch.zeros_like(m.wr)
    m.wr[1::2] = -0.0  # logits of 0 and -0
    r = m.run()
    np.testing.assert_array_equal(r.topk_ids.cpu().numpy(), np.tile(np.arange(k), (t, 1)))
    np.testing.assert_array_equal(r.topk_weights.cpu().numpy(), np.full((t, k), 0.2, np.float32))


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("t", [1, 5, 64])
def test_given_routing(t, fmt):
    """Ids that name no expert, an expert named twice, everyone at one expert, a token at none."""
    e, k = 6, 4
    m = Layer(t, 96, 64, e, k, fmt, torch.bfloat16, 4)
    rng = np.random.default_rng(5)
    ids = rng.integers(-2, e + 2, (t, k)).astype(np.int32)
    ids[:, 0] = 3
    ids[t // 2] = [5, 5, 5, 2]
    ids[t - 1] = [-1, e, 2147483647, -2147483648]
    p = rng.standard_normal((t, k)).astype(np.float32)
    r = m.run(topk_ids=dev(ids), topk_weights=dev(p))
    m.check(r, ids.astype(np.int64), p.astype(np.float64), np.abs(p) * 4 * U)
    assert torch.equal(r.y[t - 1], torch.zeros_like(r.y[t - 1]))


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_an_infinity_stays_with_its_token(fmt):
    m = Layer(4, 96, 64, 6, 2, fmt, torch.float32, 6)
    clean = m.run()
    m.x[2, 5] = float("inf")
    r = m.run(topk_ids=clean.topk_ids, topk_weights=clean.topk_weights)
    keep = [0, 1, 3]
    assert torch.equal(r.y[keep], clean.y[keep]) and not torch.isfinite(r.y[2]).all()
    m.x[2] = float("nan")
    ids = m.run().topk_ids  # unspecified experts, but experts
    assert int(ids.min()) >= 0 and int(ids.max()) < 6


def test_mx_scales_over_the_whole_exponent_range():
    # E8M0 bytes from 2^-127 up to where 6 * 2^(b - 127) is still a binary32 number.  A sum whose
    # terms reach below 2^-126 is rounded to multiples of 2^-149 at each of them.
    t, d, i = 3, 64, 96
    m = Layer(t, d, i, 1, 1, "mxfp4", torch.float32, 8)
    old = m.w2.scales.cpu().numpy().astype(np.int64)
    new = np.resize(np.array([0, 1, 2, 60, 127, 200, 245]), d)[:, None] + np.zeros_like(old)
    m.v2 = m.v2 * 2.0 ** np.repeat(new - old, 32, axis=1)
    m.w2.scales = dev(new.astype(np.uint8))
    ids, p, dp = m.routing()
    y, dy = m.reference(ids, p, dp, True)
    err = np.abs(m.run().y.double().cpu().numpy() - y)
    assert np.all(err <= dy + (3 * i + 24) * 2.0 ** -149)


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_a_nan_weight_stays_in_its_row(fmt):
    m = Layer(5, 64, 96, 4, 2, fmt, torch.bfloat16, 9)
    clean = m.run()
    e, row = int(clean.topk_ids[1, 0]), 37
    if fmt == "fp8":
        m.w2.codes.view(torch.uint8)[e * 64 + row, 11] = 0x7F
    else:
        m.w2.scales[e * 64 + row, 1] = 255 if fmt == "mxfp4" else 0x7F
    y = m.run().y
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[(clean.topk_ids == e).any(1), row] = True
    assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], clean.y[~hit])


def test_same_bits_again_in_a_graph_and_on_another_stream():
    m = Layer(20, 256, 96, 16, 4, "nvfp4", torch.bfloat16, 7)
    x, wr = m.x.to(DEV), m.wr.to(DEV)
    call = lambda out=None: fq.moe_layer(x, m.w13, m.w2, 16, 4, router=wr, out=out)
    first = call()
    for _ in range(3):
        r = call()
        assert torch.equal(r.y, first.y) and torch.equal(r.topk_weights, first.topk_weights)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        y2 = call().y
        out = torch.empty_like(first.y)
        call(out)
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            call(out)
    torch.cuda.synchronize()
    assert torch.equal(y2, first.y)
    for _ in range(3):
        out.zero_()
        graph.replay()
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, first.y)


def test_no_tokens_and_refusals():
    m = Layer(4, 64, 32, 6, 2, "mxfp4", torch.bfloat16, 8)
    x, wr = m.x.to(DEV), m.wr.to(DEV)
    r = fq.moe_layer(x[:0], m.w13, m.w2, 6, 2, router=wr)
    assert r.y.shape == (0, 64) and r.topk_ids.shape == (0, 2)
    call = lambda x=x, w13=m.w13, w2=m.w2, e=6, k=2, **kw: fq.moe_layer(x, w13, w2, e, k, **{"router": wr, **kw})
    with pytest.raises(fq.Fp4qError, match="tokens"):
        call(x=torch.zeros(65, 64, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(fq.Fp4qError, match="top_k"):
        call(k=7)
    with pytest.raises(fq.Fp4qError, match="top_k"):
        call(k=0)
    with pytest.raises(ValueError, match="topk_ids and topk_weights"):
        call(router=None)
    with pytest.raises(ValueError, match="router must"):
        call(router=wr[:5].contiguous())
    with pytest.raises(ValueError, match="w13"):
        call(e=7)
    with pytest.raises(ValueError, match="w2"):
        call(w2=m.w13)
    with pytest.raises(ValueError, match="one format"):
        call(w2=fq.ExpertWeights(fq.FMT_UE4M3, m.w2.codes, m.w2.scales))
    with pytest.raises(ValueError, match="fmt"):
        call(w13=fq.ExpertWeights(2, m.w13.codes, m.w13.scales), w2=fq.ExpertWeights(2, m.w2.codes, m.w2.scales))
    with pytest.raises(TypeError):
        call(w13=fq.ExpertWeights(fq.FMT_MXFP4, m.w13.codes, m.w13.scales.float()))
    with pytest.raises(ValueError, match="topk_ids must"):
        call(router=None, topk_ids=torch.zeros(4, 2, dtype=torch.int64, device=DEV), topk_weights=torch.zeros(4, 2, device=DEV))
    with pytest.raises(fq.Fp4qError, match="UE4M3 only"):
        call(w13=fq.ExpertWeights(fq.FMT_MXFP4, m.w13.codes, m.w13.scales, torch.ones(1, device=DEV)))
    with pytest.raises(fq.Fp4qError, match="workspace"):
        call(ws=torch.zeros(256, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_weights_past_32_bits(fmt):
    """Stacked weights of over 2^31 bytes: the last expert gives what it gives alone."""
    d, i = 4096, 2048
    m = Layer(3, d, i, 1, 1, fmt, torch.bfloat16, 10)
    per = m.w13.codes.numel()
    e = (1 << 31) // per + 2
    def stack(w):
        codes = torch.zeros(e * w.codes.shape[0], w.codes.shape[1], dtype=torch.uint8, device=DEV)
        codes[-w.codes.shape[0]:] = w.codes.view(torch.uint8)
        scales = w.scales.new_zeros(e * w.scales.shape[0], w.scales.shape[1])
        scales[-w.scales.shape[0]:] = w.scales
        return fq.ExpertWeights(w.fmt, codes.view(w.codes.dtype), scales, w.g)
    ids = torch.full((3, 1), e - 1, dtype=torch.int32, device=DEV)
    wts = torch.ones(3, 1, device=DEV)
    got = fq.moe_layer(m.x.to(DEV), stack(m.w13), stack(m.w2), e, 1, topk_ids=ids, topk_weights=wts).y
    ids0 = torch.zeros_like(ids)
    want = fq.moe_layer(m.x.to(DEV), m.w13, m.w2, 1, 1, topk_ids=ids0, topk_weights=wts).y
    assert (got.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max() and got.any()
