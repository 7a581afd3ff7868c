"""GPU: the block-scaled FP8 matrix product against the same product in 64 bits.

The tolerance is the error bound of the operation, not a fit.  With
S = sum_k |a_k b_k| (scaled), binary32 sums of 128 products and of K/128
blocks in any order, truncated or rounded, are off by at most
(128 + K/128 + 4) * 2^-23 * S (the 4 covers the scale product, its
multiplications and the conversions), and a BF16 output by half a unit in its
last place more, 2^-8 of its value."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_quantization_gb300 as m
    m.abi()
    return m


def codes(shape, gen):
    """E4M3 codes of N(0, 32) values: normal, subnormal and saturated ones."""
    x = (32.0 * torch.randn(shape, device="cuda", generator=gen)).clamp(-448, 448)
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def values(c):
    return c.view(torch.float8_e4m3fn).double()


def scales(shape, gen):
    return torch.exp(torch.randn(shape, device="cuda", generator=gen))


def expand_rows(c, s):
    M, K = c.shape
    return (values(c).view(M, K // 128, 128) * s.double()[..., None]).view(M, K)


def expand_weight(c, s):
    N, K = c.shape
    rows = torch.arange(N, device="cuda") // (1 if s.shape[0] == N else 128)
    return expand_rows(c, s[rows])


def check(out, a, b, K):
    """out against a @ b.T in 64 bits, elementwise, within the bound."""
    ref = a @ b.t()
    tol = (128 + K // 128 + 4) * 2.0 ** -23 * (a.abs() @ b.abs().t())
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ref.abs()
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol.clamp(min=1e-300)).max())} of the bound"


def make(M, N, K, G, rows, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lead = () if G is None else (G,)
    y, w = codes((M, K), gen), codes((*lead, N, K), gen)
    ys = scales((M, K // 128), gen)
    ws = scales((*lead, N if rows == 1 else -(-N // 128), K // 128), gen)
    return y, ys, w, ws


SHAPES = [(1, 1, 128), (1, 8, 256), (3, 129, 128), (128, 128, 128), (129, 257, 384), (127, 255, 1024),
          (16, 2048, 896), (64, 1000, 2048), (65, 264, 640), (300, 520, 1408), (640, 1536, 256),
          (1000, 2050, 512)]


@pytest.mark.parametrize("rows", [128, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_dense(fq, shape, dtype, rows):
    M, N, K = shape
    y, ys, w, ws = make(M, N, K, None, rows, M + N + K)
    out = fq.fp8_matmul(y, ys, w, ws, out_dtype=dtype)
    assert out.dtype == dtype and out.shape == (M, N)
    check(out, expand_rows(y, ys), expand_weight(w, ws), K)


# counts per group: empty groups at the ends and inside, single rows, groups
# around the tile sizes, and rows that belong to no group (rest)
GROUPS = {
    "one": ([5], 0), "empty": ([0, 0, 7, 0], 0), "ones": ([1] * 9, 0), "none": ([0, 0], 33),
    "edges": ([127, 128, 129, 1, 0, 256, 257], 0), "rest": ([40, 0, 90, 3], 70),
    "many": ([i % 5 for i in range(70)], 1), "big_first": ([700, 2, 30, 1], 0),
}


@pytest.mark.parametrize("rows", [128, 1])
@pytest.mark.parametrize("case", sorted(GROUPS))
@pytest.mark.parametrize("N,K", [(264, 384), (128, 640), (100, 128)])
def test_groups(fq, case, rows, N, K):
    counts, rest = GROUPS[case]
    G, M = len(counts), sum(counts) + rest
    offs = np.concatenate([[0], np.cumsum(counts)])
    y, ys, w, ws = make(M, N, K, G, rows, len(case))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((M, N), float("nan"), dtype=torch.float32, device="cuda")
    fq.fp8_matmul(y, ys, w, ws, torch.from_numpy(offs).cuda(), out=out, dev_status=status)
    for g in range(G):
        lo, hi = int(offs[g]), int(offs[g + 1])
        if hi > lo:
            check(out[lo:hi], expand_rows(y[lo:hi], ys[lo:hi]), expand_weight(w[g], ws[g]), K)
    assert bool((out[int(offs[-1]):] == 0).all())
    assert int(status) == 0


@pytest.mark.parametrize("offs,meant", [([5, 60, 200], [0, 60, 200]), ([0, 300, 200], [0, 200, 200]),
                                        ([0, -4, 130], [0, 0, 130]), ([0, 90, 40], [0, 90, 90])])
def test_malformed_offsets_are_clamped(fq, offs, meant):
    M, N, K = 200, 136, 256
    y, ys, w, ws = make(M, N, K, 2, 128, 3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = fq.fp8_matmul(y, ys, w, ws, torch.tensor(offs, device="cuda"), dev_status=status)
    good = fq.fp8_matmul(y, ys, w, ws, torch.tensor(meant, device="cuda"))
    assert int(status) == 1 and torch.equal(out, good)


@pytest.mark.parametrize("M", [4, 200])
def test_nan_stays_in_its_row_and_column(fq, M):
    N, K = 264, 384
    y, ys, w, ws = make(M, N, K, None, 1, 5)
    y[2, 130] = 0x7F
    ys[3, 0] = float("nan")
    w[7, 1] = 0xFF
    ws[9, 2] = float("nan")
    out = fq.fp8_matmul(y, ys, w, ws, out_dtype=torch.float32)
    bad = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    bad[2:4] = True
    bad[:, 7] = True
    bad[:, 9] = True
    assert torch.equal(out.isnan(), bad)


def test_zero_rows_and_zero_scales(fq):
    y, ys, w, ws = make(0, 64, 128, None, 128, 1)
    assert fq.fp8_matmul(y, ys, w, ws).shape == (0, 64)
    y, ys, w, ws = make(9, 72, 256, None, 128, 1)
    assert bool((fq.fp8_matmul(y, torch.zeros_like(ys), w, ws) == 0).all())


@pytest.mark.parametrize("M,N", [(5, 40), (300, 264)])
def test_nothing_is_written_outside_the_output(fq, M, N):
    y, ys, w, ws = make(M, N, 256, None, 128, 2)
    for dtype in (torch.bfloat16, torch.float32):
        raw = torch.full((M * N + 256,), 7.0, dtype=dtype, device="cuda")
        fq.fp8_matmul(y, ys, w, ws, out=raw[128:128 + M * N].view(M, N))
        assert bool((raw[:128] == 7).all()) and bool((raw[128 + M * N:] == 7).all())


@pytest.mark.parametrize("M", [3, 520])
def test_same_bits_again_and_on_another_stream(fq, M):
    y, ys, w, ws = make(M, 1032, 1024, None, 128, 8)
    first = fq.fp8_matmul(y, ys, w, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = fq.fp8_matmul(y, ys, w, ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, other) and torch.equal(first, fq.fp8_matmul(y, ys, w, ws))


def test_quantized_operands_end_to_end(fq):
    """BF16 tensors through the library's own quantizers: the product is off
    from the BF16 one by the quantization alone (2^-4 of each factor at most,
    relative to its block's or tile's maximum; far less in the mean)."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((200, 1024), device="cuda", generator=gen).bfloat16()
    v = (0.02 * torch.randn((384, 1024), device="cuda", generator=gen)).bfloat16()
    out = fq.fp8_matmul(*fq.fp8_quantize_1x128(x), *fq.fp8_quantize_128x128(v),
                        out_dtype=torch.float32)
    ref = x.double() @ v.double().t()
    assert float((out.double() - ref).norm() / ref.norm()) < 2.0 ** -4
