"""A mixture-of-experts layer in FP8, forward and backward, with the library's calls.

    y[t] = sum_j w[t, j] W2[e] silu(W1[e] x[t]),   e = ids[t, j]

Routing (moe_route), the row order (moe_sort_rows), the expert products
(fp8_matmul on rows quantized by fp8_quantize_1x128 and weights by
fp8_quantize_128x128), the weight gradients (fp8_matmul_wgrad on columns
quantized by fp8_quantize_cols) and the router's gradient (moe_route_backward)
run in the library; torch holds the memory, gathers rows and applies the
activation.  Rows of a group follow each other without padding.

Run on a GB300 as `python examples/moe_fp8_layer.py`: prints how far the result
and the gradients are from the same layer in float32, and the step's time.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_quantization_gb300 as fq  # noqa: E402


class ExpertWeights:
    """BF16 weights [E, N, K] with their FP8 operands: for the forward product
    and, transposed, for the input gradient (the same 128x128 tiles)."""

    def __init__(self, w: torch.Tensor):
        E, N, K = w.shape
        self.w = w
        self.q, self.s = self._quantize(w)
        self.qT, self.sT = self._quantize(w.transpose(1, 2).contiguous())

    @staticmethod
    def _quantize(w):
        E, N, K = w.shape
        q, s = fq.fp8_quantize_128x128(w.view(E * N, K))
        return q.view(E, N, K), s.view(E, N // 128, K // 128)


class MoELayer:
    def __init__(self, router: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor, k: int,
                 bias: torch.Tensor | None = None, score: str = "sigmoid"):
        self.router, self.bias, self.score, self.k = router, bias, score, k
        self.w1, self.w2 = ExpertWeights(w1), ExpertWeights(w2)
        self.E = w1.shape[0]

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """BF16 [T, H] -> BF16 [T, H]; keeps what the backward pass reads."""
        logits = x.float() @ self.router.t()
        weights, ids = fq.moe_route(logits, self.k, bias=self.bias, score=self.score)
        offsets, pair, row = fq.moe_sort_rows(ids, self.E)
        token = pair // self.k
        q, s = fq.fp8_quantize_1x128(x)  # each token once, then gathered as codes
        h = fq.fp8_matmul(q[token], s[token], self.w1.q, self.w1.s, offsets)
        a = torch.nn.functional.silu(h)
        y = fq.fp8_matmul(*fq.fp8_quantize_1x128(a), self.w2.q, self.w2.s, offsets)
        y = y[row.long()]  # [T, k, H]
        self.saved = x, logits, weights, ids, offsets, pair, row, token, h, a, y
        return (y * weights.unsqueeze(-1)).sum(1).to(x.dtype)

    def backward(self, dout: torch.Tensor):
        """BF16 [T, H] -> (dx [T, H], drouter [E, H], dw1, dw2 float32)."""
        x, logits, weights, ids, offsets, pair, row, token, h, a, y = self.saved
        dweights = (dout.unsqueeze(1).float() * y.float()).sum(-1)
        dlogits = fq.moe_route_backward(logits, ids, dweights, score=self.score)
        dy = (dout[token] * weights.view(-1)[pair.long()].unsqueeze(-1)).to(dout.dtype)
        dw2 = fq.fp8_matmul_wgrad(*fq.fp8_quantize_cols(dy, offsets),
                                  *fq.fp8_quantize_cols(a, offsets), offsets)
        da = fq.fp8_matmul(*fq.fp8_quantize_1x128(dy), self.w2.qT, self.w2.sT, offsets)
        sig = torch.sigmoid(h.float())
        dh = (da * (sig * (1 + h * (1 - sig)))).to(h.dtype)
        dw1 = fq.fp8_matmul_wgrad(*fq.fp8_quantize_cols(dh, offsets),
                                  *fq.fp8_quantize_cols(x[token], offsets), offsets)
        dx = fq.fp8_matmul(*fq.fp8_quantize_1x128(dh), self.w1.qT, self.w1.sT, offsets)
        dx = dx[row.long()].float().sum(1) + dlogits @ self.router
        return dx.to(x.dtype), dlogits.t() @ x.float(), dw1, dw2


def reference(layer: MoELayer, x: torch.Tensor, dout: torch.Tensor):
    """The same layer in float32 through autograd, for the layer's own ids."""
    ids = layer.saved[3].long()
    x = x.float().requires_grad_()
    router = layer.router.clone().requires_grad_()
    w1 = layer.w1.w.float().requires_grad_()
    w2 = layer.w2.w.float().requires_grad_()
    logits = x @ router.t()
    score = torch.sigmoid(logits) if layer.score == "sigmoid" else torch.softmax(logits, 1)
    w = score.gather(1, ids)
    w = w / w.sum(1, keepdim=True)
    out = torch.zeros_like(x)
    for e in range(layer.E):
        t, j = (ids == e).nonzero(as_tuple=True)
        y = torch.nn.functional.silu(x[t] @ w1[e].t()) @ w2[e].t()
        out = out.index_add(0, t, y * w[t, j].unsqueeze(-1))
    out.backward(dout.float())
    return out.detach(), x.grad, router.grad, w1.grad, w2.grad


def make(T, H, F, E, k, score="sigmoid", seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    layer = MoELayer(randn(E, H) / H ** 0.5, (randn(E, F, H) / H ** 0.5).bfloat16(),
                     (randn(E, H, F) / F ** 0.5).bfloat16(), k,
                     bias=0.1 * randn(E) if score == "sigmoid" else None, score=score)
    return layer, randn(T, H).bfloat16(), randn(T, H).bfloat16()


def main():
    layer, x, dout = make(4096, 2048, 1024, 32, 8)
    out = layer.forward(x)
    got = (out, *layer.backward(dout))
    for name, a, b in zip(("out", "dx", "drouter", "dw1", "dw2"), got, reference(layer, x, dout)):
        print(f"{name}: {float((a.float() - b).norm() / b.norm()):.3f} off float32")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(10):
        layer.forward(x)
        layer.backward(dout)
    end.record()
    end.synchronize()
    print(f"forward + backward: {start.elapsed_time(end) / 10:.3f} ms")


if __name__ == "__main__":
    main()
