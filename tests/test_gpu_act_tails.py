"""GPU: the activations of the FP8 products' epilogues far out.  Every product here is one
code of 1 times a row's scale, so that what is activated is exactly the scale.

Where sigma(t) is small, x sigma(t) and its derivative are held to their relative error, down
to the smallest normal number.  In binary32, with ex2.approx (2 ulp: 2^-22) and rcp.approx
(1 ulp: 2^-23):
  h = 2^(-|t| log2(e) / 2): five roundings of the exponent's argument, 1.25 |t| 2^-23, and
      2^-22  =>  rel(h) <= (2 + 1.25 |t|) 2^-23,  rel(e) <= (4.5 + 2.5 |t|) 2^-23, e = h h rounded
  s: the error of e times 1 - s, 1 + e rounds (2^-24), the reciprocal (2^-23), up to three
      products (3 2^-24): rel(x s) <= ((1 - s) (4.5 + 2.5 |t|) + 3) 2^-23
  q = s (1 - s) = e r r, times x t' (six roundings more): (4.5 + 2.5 |t| + 8) 2^-23 of |q x t'|
What is below the normal numbers on the way is off by 2^-150, and is multiplied by |x t'| at
most: 2^-147 (1 + |x t'|) in all.  Beyond e = 2^-149 that is all there is to a gradient.
A result is rounded by 2^-24 or 2^-8 of its value, a subnormal one by 2^-150 or 2^-134."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

C = 2 * math.sqrt(2 / math.pi)
DTYPES = [torch.bfloat16, torch.float32]
# rows, columns, K: few rows, few rows over a cluster, tiles of one CTA and of pairs
SHAPES = [(3, 40, 256), (16, 264, 1024), (200, 1036, 256), (700, 520, 256), (9000, 1056, 2048)]
POINTS = {"silu": (-104.0, -80.0), "gelu_tanh": (-10.8, -9.0)}


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_quantization_gb300 as m
    m.abi()
    return m


def operands(x, N, K, gated):
    """Products of exactly x[m] in every column, and, gated, of 1 for the up projection."""
    M = x.numel()
    y = torch.zeros((M, K), dtype=torch.uint8, device="cuda")
    y[:, 0] = y[:, 128] = 0x38  # 1
    w = torch.zeros((*((2,) if gated else ()), N, K), dtype=torch.uint8, device="cuda")
    w[(0, slice(None), 0) if gated else (slice(None), 0)] = 0x38
    if gated:
        w[1, :, 128] = 0x38
    ys = torch.ones((M, K // 128), device="cuda")
    ys[:, 0] = x
    ws = torch.ones((*w.shape[:-2], -(-N // 128), K // 128), device="cuda")
    return y, ys, w, ws


def form(x, fn):
    """x s, its derivative and the bounds of both in 64 bits."""
    x = x.double()
    t, dt = (x, torch.ones_like(x)) if fn == "silu" else \
        (C * (x + 0.044715 * x ** 3), C * (1 + 3 * 0.044715 * x ** 2))
    s, n = torch.sigmoid(t), torch.sigmoid(-t)
    q = s * n * x * dt
    rel = (n * (4.5 + 2.5 * t.abs()) + 3) * 2.0 ** -23
    under = 2.0 ** -147 * (1 + (x * dt).abs())
    return x * s, s + q, (x * s).abs() * rel + under, s * rel + q.abs() * (12.5 + 2.5 * t.abs()) * 2.0 ** -23 + under


def rounded(v, dtype):
    return v.abs() * 2.0 ** -24 + (2.0 ** -150 if dtype == torch.float32 else
                                   2.0 ** -134 + 2.0 ** -8 * v.abs())


def check(got, want, bound):
    off = (got.double() - want[:, None]).abs()
    assert bool((off <= bound[:, None]).all()), float((off / bound[:, None]).max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("fn", sorted(POINTS))
def test_values_keep_their_relative_error(fq, fn, shape, dtype):
    M, N, K = shape
    x = torch.linspace(*POINTS[fn], M, device="cuda")
    if M < 20:  # some of them within what sigma alone would lose
        x = torch.linspace(*{"silu": (-91.5, -87.5), "gelu_tanh": (-10.09, -9.98)}[fn], M, device="cuda")
    want, _, off, _ = form(x, fn)
    off = off + rounded(want, dtype)
    y, ys, w, ws = operands(x, N, K, False)
    check(fq.fp8_matmul_act(y, ys, w, ws, act=fn, out_dtype=dtype), want, off)
    y, ys, w, ws = operands(x, N, K, True)
    check(fq.fp8_matmul_gated(y, ys, w, ws, act=fn, out_dtype=dtype), want, off + 2.0 ** -24 * want.abs())


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("fn", sorted(POINTS))
def test_gradients_keep_their_relative_error(fq, fn, shape, dtype, gated):
    M, N, K = shape
    lo, hi = POINTS[fn] if M >= 20 else {"silu": (-91.5, -87.5), "gelu_tanh": (-10.09, -9.98)}[fn]
    z = torch.linspace(lo, hi, M, device="cuda").bfloat16()
    a, slope, da, ds = form(z, fn)
    y, ys, w, ws = operands(torch.ones(M, device="cuda"), N, K, False)  # the gradient of every value is 1
    zz = z[:, None].expand(M, N)
    zz = torch.stack((zz, torch.ones_like(zz)), 1) if gated else zz.contiguous()
    h = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    dz = fq.fp8_matmul_act_backward(y, ys, w, ws, zz, act=fn, h=h, out_dtype=dtype)
    check(dz[:, 0] if gated else dz, slope, ds + 2.0 ** -23 * slope.abs() + rounded(slope, dtype))
    if gated:
        check(dz[:, 1], a, da + 2.0 ** -24 * a.abs() + rounded(a, dtype))
    check(h, a, da + 2.0 ** -24 * a.abs() + rounded(a, torch.bfloat16))


SPECIAL = [0.0, -0.0, 1e-30, -1e-30, 1e-37, -1e-37, 20.0, -20.0, 104.0, -104.0, 200.0, -200.0, 1e4, -1e4, 1e10,
           -1e10, 1e19, -1e19, 3e38, -3e38, float("inf"), float("-inf"), float("nan")]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M", [23, 230, 9200])
@pytest.mark.parametrize("fn", ["none", "relu", "silu", "gelu_tanh"])
def test_limits_of_the_forward_activation(fq, fn, M, dtype):
    """-inf gives 0 (without an activation -inf), +inf stays, NaN stays in its row; large values
    are themselves or 0, small ones half of themselves."""
    N, K = 1056, 2048
    x = torch.tensor(SPECIAL * (M // len(SPECIAL)), device="cuda")
    y, ys, w, ws = operands(x, N, K, False)
    bias = torch.zeros(N, device="cuda")
    z = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    out = fq.fp8_matmul_act(y, ys, w, ws, bias=bias, act=fn, z=z, out_dtype=dtype)
    nan = x.isnan()
    assert torch.equal(out.isnan(), nan[:, None].expand(M, N))
    assert torch.equal(z[~nan], x[~nan].bfloat16()[:, None].expand(-1, N))
    if fn == "none":
        want = x
    elif fn == "relu":
        want = torch.where(x > 0, x, torch.zeros_like(x))
    else:
        want = torch.where(x >= 200, x, torch.where(x <= -200, torch.zeros_like(x), x))
    if fn in ("none", "relu"):
        sure = ~nan
    else:
        sure = ~nan & ((x.abs() >= 200) | (x == 0))
    assert torch.equal(out[sure], want[sure].to(dtype)[:, None].expand(-1, N))
    if fn in ("silu", "gelu_tanh"):
        rest = ~nan & ~sure
        t = x[rest].double() if fn == "silu" else C * (x[rest].double() + 0.044715 * x[rest].double() ** 3)
        half = x[rest].double() * torch.sigmoid(t)
        n = torch.sigmoid(-t)
        off = half.abs() * (n * (4.5 + 2.5 * t.abs()) + 3) * 2.0 ** -23 + 2.0 ** -147 * (1 + x[rest].double().abs() ** 3)
        check(out[rest], half, off + rounded(half, dtype))
