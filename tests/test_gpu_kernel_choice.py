"""GPU: products at sizes where the choice between kernels is close, against their 64-bit
forms within derived bounds (ffn_forms): whichever runs, the result is right."""
import pytest
import torch

import ffn_forms as ff

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_quantization_gb300 as m
    m.abi()
    return m


@pytest.mark.parametrize("M,N,K,G", [(64, 1024, 2048, 4), (64, 1024, 1024, 8), (300, 1408, 2048, 7)])
def test_ragged_rows_whose_k_may_be_split(fq, M, N, K, G):
    cut = torch.randint(0, M + 1, (G - 1,), generator=torch.Generator().manual_seed(N)).sort().values
    bounds = [0, *cut.tolist(), M]
    y, ys, w, ws, gen = ff.make(M, N, K, G, 128, M + N, ())
    offs = torch.tensor(bounds, device="cuda")
    x, off = ff.product(y, ys, w, ws, bounds)
    a, _, da, _ = ff.act(x, "silu")
    for dtype in (torch.bfloat16, torch.float32):
        out = fq.fp8_matmul_act(y, ys, w, ws, offs, act="silu", out_dtype=dtype)
        ff.check("act", out, a, da + ff.SLOPE * off + ff.rounded(a, dtype))


@pytest.mark.parametrize("M,F,K", [(64, 2048, 20480), (384, 2048, 20480), (384, 14336, 4096), (640, 13824, 5120)])
def test_dense_gated_projections_of_large_weights(fq, M, F, K):
    """More than 64 MB of weights: tiles of one CTA or of pairs, by their rounds over the SMs."""
    y, ys, w, ws, _ = ff.make(M, F, K, None, 128, M + F, (2,))
    gate, dg = ff.product(y, ys, w[0], ws[0])
    up, du = ff.product(y, ys, w[1], ws[1])
    a, _, da, _ = ff.act(gate, "silu")
    da = da + ff.SLOPE * dg
    want, off = a * up, da * (up.abs() + du) + a.abs() * du
    z = torch.empty((M, 2, F), dtype=torch.bfloat16, device="cuda")
    h = fq.fp8_matmul_gated(y, ys, w, ws, z=z, out_dtype=torch.float32)
    ff.check("h", h, want, off + ff.rounded(want, torch.float32))
    ff.check("gate", z[:, 0], gate, dg + ff.rounded(gate, torch.bfloat16))
    ff.check("up", z[:, 1], up, du + ff.rounded(up, torch.bfloat16))


@pytest.mark.parametrize("M,N,K,G", [(1003, 1001, 1408, 8), (418, 2688, 1152, 2), (246, 2432, 4992, 1),
                                     (1096, 1497, 896, 7), (17, 300, 3584, 60)])
def test_small_weights(fq, M, N, K, G):
    """Every kind of epilogue where few rows, one CTA and pairs are close to one another."""
    cut = torch.randint(0, M + 1, (G - 1,), generator=torch.Generator().manual_seed(K)).sort().values
    bounds = [0, *cut.tolist(), M]
    offs = torch.tensor(bounds, device="cuda")
    y, ys, w, ws, gen = ff.make(M, N, K, G, 1, M + N, (2,))
    gate, dg = ff.product(y, ys, w[:, 0], ws[:, 0], bounds)
    up, du = ff.product(y, ys, w[:, 1], ws[:, 1], bounds)
    a, _, da, _ = ff.act(gate, "gelu_tanh")
    da = da + ff.SLOPE * dg
    want = a * up
    h = fq.fp8_matmul_gated(y, ys, w, ws, offs, act="gelu_tanh", out_dtype=torch.float32)
    ff.check("h", h, want, da * (up.abs() + du) + a.abs() * du + ff.rounded(want, torch.float32))
    one, ones = w[:, 0].contiguous(), ws[:, 0].contiguous()
    z = torch.randn((M, 2, N), device="cuda", generator=gen).bfloat16()
    dz = fq.fp8_matmul_act_backward(y, ys, one, ones, z, offs, out_dtype=torch.float32)
    s, slope, ds, dslope = ff.act(z[:, 0], "silu")
    v = z[:, 1].double()
    want = gate * v * slope
    ff.check("dgate", dz[:, 0], want, v.abs() * (dg * (slope.abs() + dslope) + gate.abs() * dslope)
             + 2.0 ** -23 * want.abs() + ff.rounded(want, torch.float32))
    want = gate * s
    ff.check("dup", dz[:, 1], want, dg * (s.abs() + ds) + gate.abs() * ds + ff.rounded(want, torch.float32))
