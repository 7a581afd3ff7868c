"""GPU: the mixture-of-experts calls together (the example layer), inside a CUDA
graph, and on tensors whose offsets pass 32 bits."""
import os
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_quantization_gb300 as m
    m.abi()
    return m


@pytest.fixture(scope="module")
def example(fq):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import moe_fp8_layer
    return moe_fp8_layer


@pytest.mark.parametrize("T,H,F,E,k,score", [(1, 256, 128, 8, 2, "sigmoid"), (37, 256, 384, 8, 3, "softmax"),
                                             (600, 512, 256, 12, 4, "sigmoid")])
def test_layer_against_float32(example, T, H, F, E, k, score):
    """E4M3's rounding is off by at most 2^-4 of an element, 2^-4 / sqrt(3) in the
    mean square; the errors of the quantized factors that a result depends on
    add up to at most that times their number (4 for the output and dw2, 6 for
    the input gradient and dw1).  The router's gradient is a difference of such
    results that may cancel to any degree, so it has no such bound: its own tests
    are those of moe_route_backward."""
    layer, x, dout = example.make(T, H, F, E, k, score, seed=T)
    out = layer.forward(x)
    got = (out, *layer.backward(dout))
    for name, a, b, n in zip(("out", "dx", "drouter", "dw1", "dw2"), got,
                             example.reference(layer, x, dout), (4, 6, None, 6, 4)):
        assert a.shape == b.shape and bool(torch.isfinite(a.float()).all()), name
        if n is None:
            continue
        off = float((a.float() - b).norm() / b.norm())
        assert off <= n * 2.0 ** -4 / 3 ** 0.5, (name, off)


def test_calls_replay_in_a_cuda_graph(fq):
    T, E, k, H, F = 96, 8, 2, 256, 384
    gen = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    w = randn(E * F, H).bfloat16()
    wq, ws = fq.fp8_quantize_128x128(w)
    wq, ws = wq.view(E, F, H), ws.view(E, F // 128, H // 128)
    many = torch.randint(-1, E, (9000,), device="cuda", generator=gen, dtype=torch.int32)

    def calls(logits, x):
        weights, ids = fq.moe_route(logits, k)
        offs, pair, row = fq.moe_sort_rows(ids, E)
        big = fq.moe_sort_rows(many, E)
        token = pair // k
        rows = x[token]
        q, s = fq.fp8_quantize_1x128(rows)
        y = fq.fp8_matmul(q, s, wq, ws, offs)
        dense = fq.fp8_matmul(q, s, wq[0], ws[0])
        a, b = fq.fp8_quantize_cols(y, offs), fq.fp8_quantize_cols(rows, offs)
        dw = fq.fp8_matmul_wgrad(*a, *b, offs)
        dl = fq.moe_route_backward(logits, ids, weights)
        return [weights, ids, offs, pair, row, *big, y, dense, *a, *b, dw, dl]

    inputs = [(randn(T, E), randn(T, H).bfloat16()) for _ in range(2)]
    logits, x = inputs[0][0].clone(), inputs[0][1].clone()
    calls(logits, x)  # lazy set-up outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = calls(logits, x)
    for l, v in inputs:
        logits.copy_(l)
        x.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(captured, calls(l, v))):
            assert torch.equal(a, b), i


def test_matmul_past_32_bit_offsets(fq):
    """300000 x 8192 outputs: 2.46 G elements, 4.9 GB."""
    M, N, K = 300000, 8192, 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    y = torch.randint(0, 120, (M, K), device="cuda", generator=gen, dtype=torch.uint8)
    w = torch.randint(0, 120, (N, K), device="cuda", generator=gen, dtype=torch.uint8)
    ys = torch.rand((M, 1), device="cuda", generator=gen)
    ws = torch.rand((N // 128, 1), device="cuda", generator=gen)
    out = fq.fp8_matmul(y, ys, w, ws)
    for lo in (0, 262144 - 5, M - 200):  # element 2^31 is in row 262144
        part = fq.fp8_matmul(y[lo:lo + 200].clone(), ys[lo:lo + 200].clone(), w, ws)
        assert torch.equal(out[lo:lo + 200], part)


def test_quantize_cols_past_32_bit_offsets(fq):
    M, K = 2200000, 1024
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((M, K), device="cuda", generator=gen, dtype=torch.bfloat16)
    yT, s = fq.fp8_quantize_cols(x)
    lo = (M // 128 - 1) * 128
    part, sp = fq.fp8_quantize_cols(x[lo:].clone())
    assert torch.equal(yT[:, lo:], part)
    assert torch.equal(s[lo // 128:lo // 128 + sp.shape[0] - 1], sp[:-1])
    first, sf = fq.fp8_quantize_cols(x[:1280].clone())
    assert torch.equal(yT[:, :1280], first) and torch.equal(s[:10], sf[:10])


def test_wgrad_past_32_bit_offsets(fq):
    """40 x 8192 x 8192 FP32 outputs: 2.68 G elements, 10.7 GB."""
    G, N, K, M = 40, 8192, 8192, 320
    gen = torch.Generator(device="cuda").manual_seed(3)
    offs = torch.arange(G + 1, device="cuda") * (M // G)
    cap = fq.fp4_to_fp8_cols_scale_capacity(M, G)
    a = torch.randint(0, 120, (N, M), device="cuda", generator=gen, dtype=torch.uint8)
    b = torch.randint(0, 120, (K, M), device="cuda", generator=gen, dtype=torch.uint8)
    sa = torch.rand((cap, N), device="cuda", generator=gen)
    sb = torch.rand((cap, K), device="cuda", generator=gen)
    out = fq.fp8_matmul_wgrad(a, sa, b, sb, offs)
    for g in (0, 31, 32, 39):  # element 2^31 opens group 32
        lo = g * (M // G)
        cut = slice(lo, lo + M // G)
        one = fq.fp8_matmul_wgrad(a[:, cut].clone(memory_format=torch.contiguous_format), sa[g:g + 2].clone(),
                                  b[:, cut].clone(memory_format=torch.contiguous_format), sb[g:g + 2].clone())
        assert torch.equal(out[g], one[0])
