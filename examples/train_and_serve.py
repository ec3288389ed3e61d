"""Train a small language model's projection in 8 bits, then serve it with experts behind it.

    python examples/train_and_serve.py [--steps 40] [--tokens 16]

1. train   a projection dim -> dim on synthetic pairs (a fixed random target map) by
           plain gradient descent; its products, forward and backward, are fp8_linear's
2. store   the trained projection as E4M3 codes under tile scales, and the experts of a
           mixture-of-experts layer in one of three formats
3. prompt  the projection of many tokens: fp8_quantize_b128 and fp8_gemm_b128
4. decode  the same for a few tokens, and the experts on what comes out: moe_layer

Prints the loss at the start and the end, and how far each output is from the same
mathematics in float32 on the stored values.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import microscaling_fp4_quantization_amd as fq  # noqa: E402

DIM, INTER, EXPERTS, TOP_K = 896, 608, 8, 2
FORMATS = ("mxfp4", "nvfp4", "e4m3")


def randn(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def train(steps, tokens):
    """(weight, losses): gradient descent of mean |x W^T - x T^T|^2 / 2 on fresh x each step."""
    target = randn(1, DIM, DIM, dtype=torch.float32) * DIM ** -0.5
    w = torch.zeros(DIM, DIM, device="cuda", requires_grad=True)
    losses = []
    for step in range(steps):
        x = randn(100 + step, tokens, DIM, dtype=torch.float32)
        err = fq.fp8_linear(x, w) - x @ target.T
        loss = err.square().sum() / (2 * tokens)
        grad, = torch.autograd.grad(loss, w)
        with torch.no_grad():
            w -= 0.3 * grad
        losses.append(loss.detach())
    return w.detach().to(torch.bfloat16), [float(v) / DIM for v in losses]


def tile_values(codes, scales):
    s = scales.repeat_interleave(128, 0)[:codes.shape[0]].repeat_interleave(128, 1)[:, :codes.shape[1]]
    return codes.float() * s


def row_values(codes, scales):
    return codes.float() * scales.t().repeat_interleave(128, 1)[:, :codes.shape[1]]


def store_experts(w, fmt):
    """ExpertWeights of a stacked matrix, and its stored values in float32."""
    if fmt == "mxfp4":
        q = fq.mxfp4_quantize(w, block_mse=False, stats=False)
        return (fq.ExpertWeights(fq.FMT_MXFP4, q.codes, q.scales),
                fq.fp4_dequantize(q.codes, q.scales, fq.FMT_MXFP4, 32))
    if fmt == "nvfp4":
        q = fq.nvfp4_quantize(w, 16, gmode=fq.G_DYNAMIC, block_mse=False, stats=False)
        return (fq.ExpertWeights(fq.FMT_UE4M3, q.codes, q.scales, q.g),
                fq.fp4_dequantize(q.codes, q.scales, fq.FMT_UE4M3, 16, g=q.g))
    q = fq.fp8_quantize_b128(w, fq.B128_TILE)
    return fq.ExpertWeights(fq.FMT_E4M3_B128, q.codes, q.scales), tile_values(q.codes, q.scales)


def project(x, q):
    """x W^T on the stored projection."""
    a = fq.fp8_quantize_b128(x)
    return fq.fp8_gemm_b128(a.codes, a.scales, q.codes, q.scales, out_dtype=torch.bfloat16), a


def off(got, want):
    return float((got.float() - want).norm() / want.norm())


def serve(weight, tokens, fmt):
    """Relative errors of (prompt projection, decode projection, expert layer)."""
    q = fq.fp8_quantize_b128(weight, fq.B128_TILE)
    wv = tile_values(q.codes, q.scales)
    errors = []
    for n in (1024, tokens):
        y, a = project(randn(n, n, DIM), q)
        errors.append(off(y, row_values(a.codes, a.scales) @ wv.T))
    w13, v13 = store_experts(randn(2, EXPERTS * 2 * INTER, DIM) * DIM ** -0.5, fmt)
    w2, v2 = store_experts(randn(3, EXPERTS * DIM, INTER) * INTER ** -0.5, fmt)
    out = fq.moe_layer(y, w13, w2, EXPERTS, TOP_K, router=randn(4, EXPERTS, DIM) * DIM ** -0.5)
    g, u = (y.float() @ v13.T).view(tokens, EXPERTS, 2, INTER).unbind(2)
    h = torch.nn.functional.silu(g) * u
    every = torch.stack([h[:, e] @ v2[e * DIM:(e + 1) * DIM].T for e in range(EXPERTS)], 1)
    ids = out.topk_ids.long()
    picked = every.gather(1, ids[:, :, None].expand(-1, -1, DIM))
    errors.append(off(out.y, (picked * out.topk_weights[:, :, None]).sum(1)))
    return errors


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=40)
    p.add_argument("--tokens", type=int, default=16, help="tokens decoded at once, at most 64")
    args = p.parse_args()
    weight, losses = train(args.steps, 2048)
    print(f"loss per output: {losses[0]:.4f} at the start, {losses[-1]:.6f} after {args.steps} steps")
    for fmt in FORMATS:
        prompt, decode, experts = serve(weight, args.tokens, fmt)
        print(f"experts in {fmt}: projection off by {prompt:.1e} (1024 tokens) and {decode:.1e} "
              f"({args.tokens}); experts by {experts:.1e}")


if __name__ == "__main__":
    main()
