"""Calls without a workspace of the caller's: in graphs, beside each other and from
several threads, each gives the bits that it gives alone."""
import threading

import pytest
import torch

import microscaling_fp4_quantization_amd as fq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def moe_case(tokens, dim, inter, experts, top_k, seed):
    """A layer in 8 bits and a call of it."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda r, c: torch.randn(r, c, generator=g, device=DEV) * c ** -0.5
    q = lambda w: fq.fp8_quantize_b128(w, fq.B128_TILE)
    w13, w2 = q(rnd(experts * 2 * inter, dim)), q(rnd(experts * dim, inter))
    w13, w2 = (fq.ExpertWeights(fq.FMT_E4M3_B128, w.codes, w.scales) for w in (w13, w2))
    router, x = rnd(experts, dim) * 4, rnd(tokens, dim) * dim ** 0.5
    return lambda **kw: fq.moe_layer(x, w13, w2, experts, top_k, router=router, **kw)


def test_graphs_of_several_sizes_on_a_stream_that_nothing_warmed_up():
    """Captured largest first, replayed smallest first, before anything else ran on their stream."""
    cases = [moe_case(t, 256, 96, 16, 4, t) for t in (40, 9, 1)]
    want = [c().y for c in cases]
    outs = [torch.zeros_like(w) for w in want]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = []
    for case, out in zip(cases, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            case(out=out)
    for _ in range(3):
        for i in (2, 1, 0, 1):
            outs[i].zero_()
            graphs[i].replay()
            cases[i]()
            torch.cuda.synchronize()
            assert torch.equal(outs[i], want[i])
    with torch.cuda.stream(side):  # an eager call on the stream that captured
        assert torch.equal(cases[1]().y, want[1])
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[1], want[1])


def test_a_graph_outlives_a_larger_call_on_its_stream():
    small, large = moe_case(3, 256, 96, 16, 4, 1), moe_case(64, 2048, 512, 16, 4, 2)
    want, want_large = small().y, large().y
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        small()
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            small(out=out)
        large()
        held = [torch.full((1 << 20,), 0x55, dtype=torch.uint8, device=DEV) for _ in range(8)]
        for _ in range(3):
            out.zero_()
            graph.replay()
            assert torch.equal(large().y, want_large)
            assert torch.equal(out, want)
    assert all(bool((h == 0x55).all()) for h in held)


def test_experts_from_two_threads_on_one_stream():
    cases = [moe_case(t, 512, 128, 32, 4, 10 + t) for t in (1, 24)]
    want = [c().y for c in cases]
    torch.cuda.synchronize()
    run_threads([(lambda c=c: c().y) for c in cases], want)


def linear_case(tokens, n, k, seed):
    """A training step of a layer: y, dx and dw in one tensor."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x, w, dy = rnd(tokens, k), rnd(n, k), rnd(tokens, n)

    def call():
        a, b = x.detach().requires_grad_(), w.detach().requires_grad_()
        y = fq.fp8_linear(a, b)
        return torch.cat([t.flatten() for t in (y.detach(), *torch.autograd.grad(y, (a, b), dy))])

    return call


def gemm_cases():
    """Products that split K, so that they need a workspace: 8-bit, MXFP4 and NVFP4."""
    g = torch.Generator(device=DEV).manual_seed(5)
    rnd = lambda m, k: torch.randn(m, k, generator=g, device=DEV)
    a, b = rnd(100, 8192), rnd(256, 8192)
    qa, qb = fq.fp8_quantize_b128(a), fq.fp8_quantize_b128(b, fq.B128_TILE)
    ma, mb = fq.mxfp4_quantize(a), fq.mxfp4_quantize(b)
    na, nb = fq.nvfp4_quantize(a), fq.nvfp4_quantize(b)
    assert fq.lib().fp8_gemm_b128_workspace_bytes(100, 256, 8192, fq.F32) > 0
    assert fq.lib().fp4_gemm_workspace_bytes(100, 256, 8192) > 0
    assert fq.lib().fp4_gemm_nvfp4_workspace_bytes(100, 256, 8192) > 0
    return [lambda: fq.fp8_gemm_b128(qa.codes, qa.scales, qb.codes, qb.scales),
            lambda: fq.fp4_gemm_mxfp4(ma.codes, ma.scales, mb.codes, mb.scales),
            lambda: fq.fp4_gemm_nvfp4(na.codes, na.scales, na.g, nb.codes, nb.scales, nb.g)]


def test_linear_layers_from_two_threads_on_one_stream():
    cases = [linear_case(70, 1000, 600, 3), linear_case(300, 200, 500, 4)]
    want = [c() for c in cases]
    torch.cuda.synchronize()
    run_threads(cases, want, 100)


def test_products_from_three_threads_on_one_stream():
    cases = gemm_cases()
    want = [c() for c in cases]
    torch.cuda.synchronize()
    run_threads(cases, want)


@pytest.mark.parametrize("which", [0, 1, 2])
def test_a_captured_product_outlives_a_larger_one(which):
    case, step = gemm_cases()[which], linear_case(4096, 1024, 4096, 6)
    want = case()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        case()
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out = case()
        step()
        held = [torch.full((1 << 20,), 0x55, dtype=torch.uint8, device=DEV) for _ in range(8)]
        for _ in range(3):
            out.zero_()
            graph.replay()
            step()
            assert torch.equal(out, want)
    assert all(bool((h == 0x55).all()) for h in held)


def quantize_cases():
    """Calls whose later launches read what the earlier ones left in their workspace: the
    per-tensor scale and the error sums."""
    g = torch.Generator(device=DEV).manual_seed(7)
    xs = [torch.randn(m, 4096, generator=g, device=DEV) * s for m, s in ((64, 1.0), (300, 50.0))]

    def call(x):
        q = fq.nvfp4_quantize(x)
        m, n = fq.fp4_quantize_mx_nv(x)
        return torch.cat([q.g, n.g, q.stats.float(), m.stats.float(), n.stats.float(), q.codes.flatten().float()])

    return [lambda x=x: call(x) for x in xs]


def test_quantizers_from_two_threads_on_one_stream():
    cases = quantize_cases()
    want = [c() for c in cases]
    torch.cuda.synchronize()
    run_threads(cases, want)


def test_captured_quantizers_beside_eager_ones():
    """A graph on one stream, eager calls of another tensor on the stream that captured it."""
    small, large = quantize_cases()
    want, want_large = small(), large()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = small()
    for _ in range(20):
        with torch.cuda.stream(other):
            graph.replay()
        with torch.cuda.stream(side):
            got = large()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(got, want_large)


def run_threads(calls, want, rounds=200):
    """Each call over and over from a thread of its own, all on the current stream."""
    stream, bad = torch.cuda.current_stream(), []
    start = threading.Barrier(len(calls))

    def work(i):
        try:
            with torch.cuda.stream(stream):
                start.wait()
                got = [calls[i]() for _ in range(rounds)]
                bad.extend(i for g in got if not torch.equal(g, want[i]))
        except Exception as e:  # noqa: BLE001 (told to the main thread)
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:3]
