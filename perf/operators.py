"""Performance cases of the 8-bit block-128 and mixture-of-experts operators.

Four operators of a quantized language model's linear layers:

  quantize  E4M3 codes with one binary32 scale per 128 elements, of a matrix
            and of its transpose (``fp8_quantize_b128``)
  gemm      the product of two such operands (``fp8_gemm_b128``)
  linear    a training step's linear layer on them: y, dx and dw (``fp8_linear``)
  moe       a mixture-of-experts layer for a few tokens on MXFP4, NVFP4 or
            E4M3 block-128 weights (``moe_layer``)

Definitions (RN32 is round to nearest even in binary32):

  scale     s = max(RN32(amax / 448), 2^-126) of a block: 128 consecutive
            elements of a row ("row"), or a 128 x 128 tile ("tile"); the last
            block of a row or column is shorter when the size is no multiple
  code      RN32(x / s) rounded to the nearest E4M3 value, ties to even; rows of
            codes are zero-padded to whole 16 bytes
  gemm      C[m][n] = sum_k A[m][k] sa B[n][k] sb
  linear    y = Qr(x) Qt(w)^T, dx = Qr(dy) Qt(w), dw = Qr(dy^T) Qr(x^T), with Qr
            and Qt the dequantized values under row and tile scales
  moe       l = x Wr^T; the top_k largest l of a token (ties to the lowest
            index) with softmax weights p over them (or over all experts);
            y = sum_e p_e W2_e (silu(G_e x) * (U_e x)), [G_e; U_e] = W13_e

With ``own`` false the plain forms run: elementary torch operations in binary32,
rounded once at the end.  With ``own`` true the library's calls run.
"""
import math

import torch

own = False

DEV = "cuda:0"
MIN_SCALE = 2.0 ** -126
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------
# Cases

def listed():
    return [
        # The smallest call: a decode step's activations of Qwen2.5-0.5B, where latency counts.
        {"name": "quantize-tokens-small", "op": "quantize", "rows": 7, "cols": 896, "dtype": "bf16",
         "kind": "row", "transposed": False},
        # A training step's activations (Qwen2.5-7B hidden size, 8192 tokens): both layouts in one pass.
        {"name": "quantize-tokens-both", "op": "quantize", "rows": 8192, "cols": 3584, "dtype": "bf16",
         "kind": "row", "transposed": True},
        # A master weight in binary32 with ragged edges, tile scales, both layouts.
        {"name": "quantize-weight-ragged", "op": "quantize", "rows": 4861, "cols": 5000, "dtype": "f32",
         "kind": "tile", "transposed": True},
        # One token against the Qwen2.5-7B down projection: a pass over the weight.
        {"name": "gemm-decode", "op": "gemm", "m": 1, "n": 3584, "k": 18944, "b_kind": "tile", "out": "bf16"},
        # A short batch with odd sizes, scales per row on both sides.
        {"name": "gemm-ragged", "op": "gemm", "m": 333, "n": 1031, "k": 1008, "b_kind": "row", "out": "f32"},
        # A prompt against the Qwen2.5-7B up projection: the largest product.
        {"name": "gemm-prefill", "op": "gemm", "m": 8192, "n": 18944, "k": 3584, "b_kind": "tile", "out": "bf16"},
        # A small training step with an odd token count (Qwen2.5-0.5B up projection).
        {"name": "linear-small", "op": "linear", "tokens": 509, "n": 4864, "k": 896, "dtype": "f32"},
        # An ordinary one (Llama-3.1-8B MLP).
        {"name": "linear-step", "op": "linear", "tokens": 4096, "n": 14336, "k": 4096, "dtype": "bf16"},
        # One token, many small experts: 8 of 64 are read.
        {"name": "moe-one-token", "op": "moe", "tokens": 1, "dim": 4096, "inter": 1024, "experts": 64,
         "top_k": 8, "fmt": "mxfp4", "dtype": "bf16", "renorm": True},
        # A few tokens, small layer, binary32 activations.
        {"name": "moe-small-f32", "op": "moe", "tokens": 5, "dim": 896, "inter": 480, "experts": 12,
         "top_k": 3, "fmt": "nvfp4", "dtype": "f32", "renorm": False},
        # The largest batch of the few-token form: every expert is read.
        {"name": "moe-many-tokens", "op": "moe", "tokens": 64, "dim": 4096, "inter": 1024, "experts": 64,
         "top_k": 8, "fmt": "fp8", "dtype": "bf16", "renorm": True},
        # A few large experts (Llama-3.1-8B MLP sizes), two per token.
        {"name": "moe-large-experts", "op": "moe", "tokens": 11, "dim": 4096, "inter": 14336, "experts": 8,
         "top_k": 2, "fmt": "nvfp4", "dtype": "bf16", "renorm": True},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi, unit=1, whole=64):
    """An odd multiple of `unit` or, half of the time, of `whole` (rows of whole 16 bytes) between lo and hi."""
    u = whole if rng.random() < 0.5 and hi >= whole else unit
    return u * min(_log(rng, max(1, lo // u), hi // u) | 1, (hi // u - 1) | 1)


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "linear", "moe", "moe"])
    if op == "quantize":
        return {"op": op, "rows": _size(rng, 1, 8192), "cols": _size(rng, 64, 8192),
                "dtype": rng.choice(["bf16", "f32"]), "kind": rng.choice(["row", "tile"]),
                "transposed": rng.random() < 0.6}
    if op == "gemm":
        return {"op": op, "m": _size(rng, 1, 8192), "n": _size(rng, 64, 18944),
                "k": _size(rng, 128, 4096, 16, 128), "b_kind": rng.choice(["tile", "tile", "row"]),
                "out": rng.choice(["bf16", "f32"])}
    if op == "linear":
        return {"op": op, "tokens": _size(rng, 64, 4096), "n": _size(rng, 256, 8192), "k": _size(rng, 256, 4096),
                "dtype": rng.choice(["bf16", "bf16", "f32"])}
    experts = _log(rng, 4, 64)
    return {"op": op, "tokens": _log(rng, 1, 64), "dim": _size(rng, 512, 4096, 32, 128),
            "inter": _size(rng, 256, 1024, 32, 128), "experts": experts, "top_k": rng.randint(1, min(8, experts)),
            "fmt": rng.choice(["mxfp4", "nvfp4", "fp8"]), "dtype": rng.choice(["bf16", "bf16", "f32"]),
            "renorm": rng.random() < 0.7}


def _up(n, m):
    return (n + m - 1) // m


def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once."""
    op = case["op"]
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        outs = 2 if case["transposed"] else 1
        eb = 2 if case["dtype"] == "bf16" else 4
        scales = 4 * outs * (r * _up(c, 128) if case["kind"] == "row" else _up(r, 128) * _up(c, 128))
        return {"bytes": r * c * (eb + outs) + scales, "flops": 3 * r * c}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        kb = _up(k, 128)
        sb = kb * (n if case["b_kind"] == "row" else _up(n, 128))
        return {"bytes": (m + n) * k + 4 * (m * kb + sb) + m * n * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * m * n * k}
    if op == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        eb = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": eb * (2 * t * k + 2 * n * k + 2 * t * n), "flops": 6 * t * n * k}
    t, d, i, e, k = (case[n] for n in ("tokens", "dim", "inter", "experts", "top_k"))
    per = {"mxfp4": 0.5 + 1 / 32, "nvfp4": 0.5 + 1 / 16, "fp8": 1 + 4 / 16384}[case["fmt"]]
    eb = 2 if case["dtype"] == "bf16" else 4
    active = e * (1 - (1 - k / e) ** t)  # experts that at least one token takes, on average
    return {"bytes": active * 3 * i * d * per + eb * (e * d + 2 * t * d), "flops": 2 * t * d * (3 * k * i + e)}


# --------------------------------------------------------------------------
# Inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _activations(g, rows, cols):
    """Normal values with a spread per token and 1% of the channels ten times larger."""
    x = _randn(g, rows, cols) * torch.exp(0.5 * _randn(g, rows, 1))
    loud = torch.rand(cols, generator=g, device=DEV) < 0.01
    return x * torch.where(loud, 10.0, 1.0)


def _weights_fp8(w):
    """E4M3 codes and tile scales of (experts * rows) x cols, as a checkpoint holds them."""
    return _q_tile(w)


def _weights_fp4(w, fmt):
    """E2M1 codes (two per byte) and block scales of rows x cols."""
    block = 32 if fmt == "mxfp4" else 16
    rows, cols = w.shape
    b = w.reshape(rows, cols // block, block)
    amax = b.abs().amax(2)
    if fmt == "mxfp4":
        e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -100))) - 2
        scales, s, g = (e + 127).to(torch.uint8), _pow2(e).float(), None
    else:
        g = (w.abs().amax() / 2688).reshape(1)
        sc = (amax / (6 * g)).to(torch.float8_e4m3fn)
        scales, s = sc.view(torch.uint8), sc.float() * g
    y = b / s.clamp(min=2.0 ** -100)[..., None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    n = torch.bucketize(y.abs(), edges).to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)
    n = n.reshape(rows, cols // 2, 2)
    return (n[..., 0] | (n[..., 1] << 4)).contiguous(), scales.contiguous(), g


def _experts(g, experts, rows, cols, fmt):
    """One stacked matrix (experts * rows) x cols of Normal(0, 1/sqrt(cols)) weights, quantized."""
    if fmt == "fp8":
        c, s = _weights_fp8(_randn(g, experts * rows, cols) * cols ** -0.5)
        return {"codes": c, "scales": s, "g": None}
    c, s, gg = _weights_fp4(_randn(g, experts * rows, cols) * cols ** -0.5, fmt)
    return {"codes": c, "scales": s, "g": gg}


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    if op == "quantize":
        # Activations for row scales, a weight matrix for tile scales.
        r, c = case["rows"], case["cols"]
        x = _activations(g, r, c) if case["kind"] == "row" else _randn(g, r, c) * 0.02
        st["x"] = x.to(DTYPES[case["dtype"]])
    elif op == "gemm":
        # Operands as the quantizer leaves them: activations, and a weight or a second activation.
        m, n, k = case["m"], case["n"], case["k"]
        st["a"], st["sa"] = _q_row(_activations(g, m, k))
        if case["b_kind"] == "tile":
            st["b"], st["sb"] = _q_tile(_randn(g, n, k) * 0.02)
        else:
            st["b"], st["sb"] = _q_row(_activations(g, n, k))
    elif op == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        dt = DTYPES[case["dtype"]]
        st["x"] = _activations(g, t, k).to(dt).requires_grad_()
        st["w"] = (_randn(g, n, k) * 0.02).to(dt).requires_grad_()
        st["dy"] = (_randn(g, t, n) * 1e-3).to(dt)
    else:
        t, d, i, e, k = (case[n] for n in ("tokens", "dim", "inter", "experts", "top_k"))
        dt = DTYPES[case["dtype"]]
        wr = (_randn(g, e, d) * d ** -0.5).to(dt)
        # Normalised hidden states, each leaning towards the experts that a trained router picks for it.
        pick = torch.rand(t, e, generator=g, device=DEV).argsort(1)[:, :k]
        lean = 4.0 + 0.7 * torch.arange(k, device=DEV, dtype=torch.float32)
        x = _randn(g, t, d) + (lean[None, :, None] * wr.float()[pick]).sum(1)
        st["x"], st["wr"] = x.to(dt), wr
        st["w13"] = _experts(g, e, 2 * i, d, case["fmt"])
        st["w2"] = _experts(g, e, d, i, case["fmt"])
    return st


# --------------------------------------------------------------------------
# Plain forms

def _pow2(e):
    """2^e for whole numbers e, exactly (torch's own power of two is rounded): the bits of a binary64 value."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _pad(x, rows, cols):
    """x with zeros up to whole multiples of rows and cols."""
    r, c = x.shape
    return torch.nn.functional.pad(x, (0, -c % cols, 0, -r % rows))


def _scale(amax):
    """max(RN32(amax / 448), 2^-126); a tensor divisor, since torch multiplies by a rounded reciprocal for a number."""
    return (amax / torch.full_like(amax, 448.0)).clamp(min=MIN_SCALE)


def _q_row(x):
    """Codes (rows x cols padded to 16) and scales (blocks x rows), one scale per 128 of a row."""
    r, c = x.shape
    b = _pad(x.float(), 1, 128).reshape(r, -1, 128)
    s = _scale(b.abs().amax(2))
    q = (b / s[..., None]).reshape(r, -1)[:, :_up(c, 16) * 16]
    return q.to(torch.float8_e4m3fn), s.t().contiguous()


def _q_tile(x):
    """Codes (rows x cols padded to 16) and scales (row blocks x column blocks), one scale per 128 x 128."""
    r, c = x.shape
    p = _pad(x.float(), 128, 128)
    b = p.reshape(p.shape[0] // 128, 128, p.shape[1] // 128, 128)
    s = _scale(b.abs().amax(dim=(1, 3)))
    q = (b / s[:, None, :, None]).reshape(p.shape)[:r, :_up(c, 16) * 16]
    return q.to(torch.float8_e4m3fn), s


def _d_row(codes, scales):
    """Dequantized values under row scales."""
    return codes.float() * scales.t().repeat_interleave(128, 1)[:, :codes.shape[1]]


def _d_tile(codes, scales):
    """Dequantized values under tile scales."""
    s = scales.repeat_interleave(128, 0)[:codes.shape[0]].repeat_interleave(128, 1)[:, :codes.shape[1]]
    return codes.float() * s


def _plain_quantize(x, kind, transposed):
    if kind == "row":
        c, s = _q_row(x)
        ct, s_t = _q_row(x.t()) if transposed else (None, None)
    else:
        c, s = _q_tile(x)
        ct, s_t = _q_tile(x.t()) if transposed else (None, None)
    return {"codes": c, "scales": s, "codes_t": ct, "scales_t": s_t}


def _plain_linear(x, w, dy):
    k, n = x.shape[1], w.shape[0]
    xq, wq, dyq = _d_row(*_q_row(x)), _d_tile(*_q_tile(w)), _d_row(*_q_row(dy))
    y = xq @ wq.t()
    dx = dyq[:, :n] @ wq[:, :k]
    dw = _d_row(*_q_row(dy.t())) @ _d_row(*_q_row(x.t())).t()
    return {"y": y.to(x.dtype), "dx": dx.to(x.dtype), "dw": dw.to(w.dtype)}


def _d_fp4(q, fmt):
    """E2M1 codes times their block scales (without the per-tensor scale)."""
    half = torch.tensor(E2M1, device=DEV)
    lut = torch.cat([half, -half])
    byte = torch.arange(256, device=DEV)
    pairs = torch.stack([lut[byte & 15], lut[byte >> 4]], 1)
    v = pairs[q["codes"].int()]
    rows = v.shape[0]
    if fmt == "mxfp4":
        s = _pow2(q["scales"].long() - 127).float()
    else:
        s = q["scales"].view(torch.float8_e4m3fn).float()
    return (v.reshape(rows, s.shape[1], -1) * s[..., None]).reshape(rows, -1)


def _d_experts(q, fmt):
    return _d_tile(q["codes"], q["scales"]) if fmt == "fp8" else _d_fp4(q, fmt)


def _plain_moe(st):
    case = st["case"]
    e, k, fmt, d, i = case["experts"], case["top_k"], case["fmt"], case["dim"], case["inter"]
    x = st["x"].float()
    t = x.shape[0]
    logits = x @ st["wr"].float().t()
    top, ids = logits.sort(dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    p = torch.exp(top - top[:, :1])
    p = p / (p.sum(1, keepdim=True) if case["renorm"] else torch.exp(logits - top[:, :1]).sum(1, keepdim=True))
    share = torch.zeros(t, e, device=DEV).scatter(1, ids, p)
    h = (x @ _d_experts(st["w13"], fmt).t()).reshape(t, e, 2, i)
    if fmt == "nvfp4":
        h = h * st["w13"]["g"]
    h = h[:, :, 0] / (1.0 + torch.exp(-h[:, :, 0])) * h[:, :, 1] * share[..., None]
    w2 = _d_experts(st["w2"], fmt).reshape(e, d, i).permute(1, 0, 2).reshape(d, e * i)
    y = h.reshape(t, e * i) @ w2.t()
    if fmt == "nvfp4":
        y = y * st["w2"]["g"]
    return {"y": y.to(st["x"].dtype), "ids": ids.int(), "weights": p}


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        return _plain_quantize(st["x"], case["kind"], case["transposed"])
    if op == "gemm":
        b = (_d_tile if case["b_kind"] == "tile" else _d_row)(st["b"], st["sb"])
        return (_d_row(st["a"], st["sa"]) @ b.t()).to(DTYPES[case["out"]])
    if op == "linear":
        return _plain_linear(st["x"].detach(), st["w"].detach(), st["dy"])
    return _plain_moe(st)


# --------------------------------------------------------------------------
# The library's calls

def _own(st):
    import microscaling_fp4_quantization_amd as fq
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        q = fq.fp8_quantize_b128(st["x"], fq.B128_ROW if case["kind"] == "row" else fq.B128_TILE,
                                 transposed=case["transposed"])
        return {"codes": q.codes, "scales": q.scales, "codes_t": q.codes_t, "scales_t": q.scales_t}
    if op == "gemm":
        return fq.fp8_gemm_b128(st["a"], st["sa"], st["b"], st["sb"],
                                fq.B128_ROW if case["b_kind"] == "row" else fq.B128_TILE,
                                out_dtype=DTYPES[case["out"]])
    if op == "linear":
        y = fq.fp8_linear(st["x"], st["w"])
        dx, dw = torch.autograd.grad(y, (st["x"], st["w"]), st["dy"])
        return {"y": y, "dx": dx, "dw": dw}
    fmt = {"mxfp4": fq.FMT_MXFP4, "nvfp4": fq.FMT_UE4M3, "fp8": fq.FMT_E4M3_B128}[case["fmt"]]
    r = fq.moe_layer(st["x"], fq.ExpertWeights(fmt, **st["w13"]), fq.ExpertWeights(fmt, **st["w2"]),
                     case["experts"], case["top_k"], router=st["wr"], renormalize=case["renorm"])
    return {"y": r.y, "ids": r.topk_ids, "weights": r.topk_weights}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# The definitions in 64 bits

def _x_pow2(e):
    return torch.tensor([2.0 ** k for k in range(-130, 131)], dtype=torch.float64, device=e.device)[e.long() + 130]


def _x_e4m3(v):
    """v (binary64) to the nearest E4M3 value, ties to even."""
    _, e = torch.frexp(v)  # v = m 2^e with m in [1/2, 1)
    step = _x_pow2((e - 1).clamp(min=-6) - 3)
    return ((v / step).round() * step).clamp(-448.0, 448.0)


def _x_quantized(x, tall):
    """Code values and the scale of each element, blocks of `tall` rows x 128 columns; x whole binary64 values."""
    r, c = x.shape
    p = torch.zeros(_up(r, tall) * tall, _up(c, 128) * 128, dtype=torch.float64, device=x.device)
    p[:r, :c] = x
    b = p.view(_up(r, tall), tall, _up(c, 128), 128)
    s = b.abs().amax(3).amax(1).div(448.0).float().double().clamp(min=2.0 ** -126)
    v = _x_e4m3((b / s[:, None, :, None]).float().double())
    return v.view(p.shape)[:r, :_up(c, 16) * 16], s


def _x_value(x, tall):
    v, s = _x_quantized(x, tall)
    full = s.repeat_interleave(tall, 0)[:v.shape[0]].repeat_interleave(128, 1)[:, :v.shape[1]]
    return (v * full)[:, :x.shape[1]]


def _x_stored(codes, scales, kind):
    """Stored codes and scales as binary64 values."""
    c = codes.to(torch.float64)
    s = scales.double() if kind == "tile" else scales.double().t()
    rows = torch.arange(c.shape[0], device=c.device) // (128 if kind == "tile" else 1)
    cols = torch.arange(c.shape[1], device=c.device) // 128
    return c * s[rows][:, cols]


def _x_experts(q, fmt, lo, n):
    """Rows lo .. lo + n of a stacked matrix of expert weights."""
    codes = q["codes"][lo:lo + n]
    if fmt == "fp8":
        rows = torch.arange(lo, lo + n, device=codes.device) // 128
        cols = torch.arange(codes.shape[1], device=codes.device) // 128
        return codes.to(torch.float64) * q["scales"].double()[rows][:, cols]
    c = torch.stack([codes & 15, codes >> 4], 2).reshape(n, -1)
    m, ex = (c & 1).double(), ((c >> 1) & 3).double()
    v = torch.where(ex == 0, m * 0.5, (1 + m * 0.5) * _x_pow2(ex - 1))
    v = torch.where(c > 7, -v, v)
    s = q["scales"][lo:lo + n]
    if fmt == "mxfp4":
        return v * _x_pow2(s.long() - 127).repeat_interleave(32, 1)
    return v * s.view(torch.float8_e4m3fn).to(torch.float64).repeat_interleave(16, 1) * q["g"].double()


def _exact_moe(st):
    case = st["case"]
    e, k, d, i, fmt = (case[n] for n in ("experts", "top_k", "dim", "inter", "fmt"))
    x = st["x"].double()
    logits = x @ st["wr"].double().t()
    ids = torch.argsort(-logits, dim=1, stable=True)[:, :k]
    prob = torch.softmax(logits, 1).gather(1, ids)
    if case["renorm"]:
        prob = prob / prob.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    for j in range(e):  # one expert's weights at a time
        who, slot = (ids == j).nonzero(as_tuple=True)
        if who.numel():
            gu = x[who] @ _x_experts(st["w13"], fmt, j * 2 * i, 2 * i).t()
            h = gu[:, :i] * torch.sigmoid(gu[:, :i]) * gu[:, i:]
            y.index_add_(0, who, (h @ _x_experts(st["w2"], fmt, j * d, d).t()) * prob[who, slot][:, None])
    return {"y": y, "ids": None, "weights": prob}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = st["x"].double()
        tall = 1 if case["kind"] == "row" else 128
        side = lambda v, s: (v.float(), (s.t() if tall == 1 else s).contiguous())
        c, s = side(*_x_quantized(x, tall))
        ct, s_t = side(*_x_quantized(x.t(), tall)) if case["transposed"] else (None, None)
        return {"codes": c, "scales": s, "codes_t": ct, "scales_t": s_t}
    if op == "gemm":
        return _x_stored(st["a"], st["sa"], "row") @ _x_stored(st["b"], st["sb"], case["b_kind"]).t()
    if op == "linear":
        x, w, dy = (st[n].detach().double() for n in ("x", "w", "dy"))
        wq = _x_value(w, 128)
        return {"y": _x_value(x, 1) @ wq.t(), "dx": _x_value(dy, 1) @ wq,
                "dw": _x_value(dy.t(), 1) @ _x_value(x.t(), 1).t()}
    return _exact_moe(st)
