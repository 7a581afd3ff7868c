"""GPU: the products of few rows over as many groups as two CTAs of an SM have room for the
offsets of, and over more, against their 64-bit forms within derived bounds (ffn_forms)."""
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


@pytest.mark.parametrize("most", [3, 24])  # rows a group: tiles of 16 rows, and of 32
@pytest.mark.parametrize("G", [371, 372, 480, 482, 1024])
def test_few_rows(fq, G, most):
    N, K = 128, 1536
    n = torch.randint(0, most + 1, (G,), generator=torch.Generator().manual_seed(G + most))
    bounds = [0] + n.cumsum(0).tolist()
    M = bounds[-1] + 5  # five rows of no group
    y, ys, w, ws, gen = ff.make(M, N, K, G, 128, G + most, (2,))
    one, ones = w[:, 0].contiguous(), ws[:, 0].contiguous()
    offs = torch.tensor(bounds, device="cuda")
    x, off = ff.product(y, ys, one, ones, bounds)
    up, off_up = ff.product(y, ys, w[:, 1], ws[:, 1], bounds)
    for dtype in (torch.bfloat16, torch.float32):
        ff.check("product", fq.fp8_matmul(y, ys, one, ones, offs, out_dtype=dtype), x,
                 off + ff.rounded(x, dtype))
    r = torch.randn((M, N), device="cuda", generator=gen)
    a, _, da, _ = ff.act(x, "silu")
    da = da + ff.SLOPE * off
    want = a + r.double()
    out = fq.fp8_matmul_act(y, ys, one, ones, offs, act="silu", residual=r, out_dtype=torch.float32)
    ff.check("act", out, want, da + 2.0 ** -24 * a.abs() + ff.rounded(want, torch.float32))
    h = fq.fp8_matmul_gated(y, ys, w, ws, offs, out_dtype=torch.float32)
    ff.check("gated", h, a * up, da * (up.abs() + off_up) + a.abs() * off_up + ff.rounded(a * up, torch.float32))
    q, s = fq.fp8_matmul_gated(y, ys, w, ws, offs, quantize=True)
    amax = h.abs().amax(1, keepdim=True)
    full = torch.full_like(amax, 448.0)
    codes = (h * (full / amax).clamp(max=3.4028234663852886e38)).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(q, codes.view(torch.uint8)) and torch.equal(s, amax / full)
