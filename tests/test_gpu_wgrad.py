"""GPU: the transposed FP8 quantizer (byte for byte against the CPU oracle's
block quantizer) and the weight-gradient product against the same product in
64 bits.

Tolerance of the product: with S = sum_t |a_t b_t| (scaled), binary32 sums
over 128 tokens and over the blocks in any order, truncated or rounded, are
off by at most (128 + blocks + 6) * 2^-23 * S (two scale products, the
addition of the previous value and the conversions in the 6); a BF16 output by
2^-8 of its value more."""
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


# counts per group and rows that belong to no group
GROUPS = {
    "one_token": ([1], 0), "empty": ([0, 0, 7, 0], 0), "no_tokens": ([0, 0, 0], 0),
    "nobody": ([0, 0], 33), "aligned": ([128, 256, 16], 0), "edges": ([127, 128, 129, 1, 0, 257], 0),
    "rest": ([40, 0, 90, 3], 70), "many": ([i % 5 for i in range(70)], 1),
    "multiple_of_16": ([100, 27, 129], 0), "big": ([700, 2, 301], 1),
}


def offsets(case):
    counts, rest = GROUPS[case]
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    return offs, int(offs[-1]) + rest


def bf16_bits(M, K, seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((M, K)) * rng.lognormal(0, 2, (M, 1))).astype(np.float32)
    t = torch.from_numpy(x).bfloat16()
    if M > 4 and K > 9:
        t[1, 3] = float("nan")
        t[2, 5] = float("inf")
        t[:, 6] = 0.0
        t[3, 7] = 3e38
        t[:, 8] = 1e-39
    return t.view(torch.int16).numpy().view(np.uint16)


def oracle_cols(oracle_mod, bits, offs, cap):
    M, K = bits.shape
    yT, sc = np.zeros((K, M), np.uint8), np.zeros((cap, K), np.float32)
    b = 0
    for lo, hi in zip(offs, offs[1:]):
        for t in range(int(lo), int(hi), 128):
            n = min(128, int(hi) - t)
            block = np.zeros((K, 128), np.uint16)
            block[:, :n] = bits[t:t + n].T
            c, s = oracle_mod.fp8_quantize_blocks(block, 1)
            yT[:, t:t + n] = c[:, :n]
            sc[b] = s[:, 0]
            b += 1
    return yT, sc


@pytest.mark.parametrize("case", sorted(GROUPS))
@pytest.mark.parametrize("K", [8, 136, 384])
def test_fp8_quantize_cols(fq, oracle_mod, case, K):
    offs, M = offsets(case)
    bits = bf16_bits(M, K, K + M)
    x = torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)
    cap = fq.fp4_to_fp8_cols_scale_capacity(M, len(offs) - 1) + 2
    raw = torch.full((K * M + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    sc = torch.full((cap, K), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    yT, got = fq.fp8_quantize_cols(x, torch.from_numpy(offs).cuda(), yT=raw[32:32 + K * M].view(K, M),
                                   yT_scale=sc, dev_status=status)
    ryT, rsc = oracle_cols(oracle_mod, bits, offs, cap)
    assert np.array_equal(yT.cpu().numpy(), ryT)
    assert np.array_equal(got.cpu().numpy().view(np.uint32), rsc.view(np.uint32))
    assert bool((raw[:32] == 0xA5).all()) and bool((raw[32 + K * M:] == 0xA5).all())
    assert int(status) == 0


def test_cols_without_offsets_is_one_group(fq):
    x = torch.randn((300, 72), device="cuda").bfloat16()
    a = fq.fp8_quantize_cols(x)
    b = fq.fp8_quantize_cols(x, torch.tensor([0, 300], device="cuda"))
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def codes(shape, gen):
    x = (32.0 * torch.randn(shape, device="cuda", generator=gen)).clamp(-448, 448)
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def values(c):
    return c.view(torch.float8_e4m3fn).double()


def operands(M, R, offs, gen, cap):
    """Transposed codes and scales; everything that belongs to no group's
    block is NaN, and must not be seen."""
    c = codes((R, M), gen)
    s = torch.exp(torch.randn((cap, R), device="cuda", generator=gen))
    c[:, int(offs[-1]):] = 0x7F
    nb = int(((np.diff(offs) + 127) // 128).sum())
    s[nb:] = float("nan")
    return c, s


def reference(a, sa, b, sb, offs):
    outs, mags, n, base = [], [], [], 0
    for lo, hi in zip(offs, offs[1:]):
        lo, hi = int(lo), int(hi)
        blk = base + torch.arange(hi - lo, device="cuda") // 128
        x = values(a[:, lo:hi].contiguous()) * sa.double()[blk].t()
        y = values(b[:, lo:hi].contiguous()) * sb.double()[blk].t()
        outs.append(x @ y.t())
        mags.append(x.abs() @ y.abs().t())
        n.append(-(-(hi - lo) // 128))
        base += n[-1]
    return torch.stack(outs), torch.stack(mags), torch.tensor(n, device="cuda").double()


def check(out, ref, mag, blocks, before=None):
    tol = (128 + blocks + 6).view(-1, 1, 1) * 2.0 ** -23 * mag
    if before is not None:
        ref = ref + before.double()
        tol = tol + 2.0 ** -22 * before.double().abs()
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ref.abs()
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol.clamp(min=1e-300)).max())} of the bound"


@pytest.mark.parametrize("case", sorted(GROUPS))
@pytest.mark.parametrize("N,K", [(1, 1), (100, 264), (257, 128), (128, 515)])
def test_wgrad(fq, case, N, K):
    offs, M = offsets(case)
    G = len(offs) - 1
    gen = torch.Generator(device="cuda").manual_seed(N + K + M)
    cap = fq.fp4_to_fp8_cols_scale_capacity(M, G)
    a, sa = operands(M, N, offs, gen, cap)
    b, sb = operands(M, K, offs, gen, cap)
    dev = torch.from_numpy(offs).cuda()
    ref, mag, blocks = reference(a, sa, b, sb, offs)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        out = fq.fp8_matmul_wgrad(a, sa, b, sb, dev, out_dtype=dtype, dev_status=status)
        assert out.shape == (G, N, K) and out.dtype == dtype
        check(out, ref, mag, blocks)
        before = torch.randn((G, N, K), device="cuda", generator=gen).to(dtype)
        again = fq.fp8_matmul_wgrad(a, sa, b, sb, dev, out=before.clone(), accumulate=True)
        check(again, ref, mag, blocks, before)
    assert int(status) == 0


@pytest.mark.parametrize("M", [1, 16, 112, 128, 1000, 1008])
def test_wgrad_of_one_group(fq, M):
    """Without offsets; M % 16 == 0 reads the operands in place."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    offs, cap = np.array([0, M]), fq.fp4_to_fp8_cols_scale_capacity(M, 1)
    a, sa = operands(M, 200, offs, gen, cap)
    b, sb = operands(M, 264, offs, gen, cap)
    ref, mag, blocks = reference(a, sa, b, sb, offs)
    check(fq.fp8_matmul_wgrad(a, sa, b, sb), ref, mag, blocks)


def test_a_nan_block_stays_in_its_group_and_row(fq):
    offs = np.array([0, 100, 210, 300])
    gen = torch.Generator(device="cuda").manual_seed(1)
    cap = fq.fp4_to_fp8_cols_scale_capacity(300, 3)
    a, sa = operands(300, 72, offs, gen, cap)
    b, sb = operands(300, 136, offs, gen, cap)
    a[5, 100:210] = 0x7F
    sa[1, 5] = float("nan")
    b[9, 209] = 0x7F
    out = fq.fp8_matmul_wgrad(a, sa, b, sb, torch.from_numpy(offs).cuda())
    bad = torch.zeros((3, 72, 136), dtype=torch.bool, device="cuda")
    bad[1, 5] = True
    bad[1, :, 9] = True
    assert torch.equal(out.isnan(), bad)


@pytest.mark.parametrize("M", [1000, 1008])
def test_operands_of_both_transposed_casts(fq, M):
    """Activations through MXFP4 (fp4_to_fp8_cols), gradients through
    fp8_quantize_cols, with the same ragged groups."""
    offs = np.array([0, 3, 3, 400, M - 60, M])
    dev = torch.from_numpy(offs).cuda()
    gen = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn((M, 256), device="cuda", generator=gen).bfloat16()
    dy = torch.randn((M, 128), device="cuda", generator=gen).bfloat16()
    b, sb = fq.fp4_to_fp8_cols(*fq.mxfp4_quantize_rows(x), dev, 3)
    a, sa = fq.fp8_quantize_cols(dy, dev)
    nb = int(((np.diff(offs) + 127) // 128).sum())
    sb[nb:] = 0  # not written by that call
    ref, mag, blocks = reference(a, sa, b, sb, offs)
    check(fq.fp8_matmul_wgrad(a, sa, b, sb, dev), ref, mag, blocks)


def test_malformed_offsets_are_clamped(fq):
    gen = torch.Generator(device="cuda").manual_seed(2)
    cap = fq.fp4_to_fp8_cols_scale_capacity(200, 2)
    a, b = codes((40, 200), gen), codes((72, 200), gen)
    sa, sb = torch.ones((cap, 40), device="cuda"), torch.ones((cap, 72), device="cuda")
    for offs, meant in (([5, 60, 200], [0, 60, 200]), ([0, 900, 100], [0, 200, 200])):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = fq.fp8_matmul_wgrad(a, sa, b, sb, torch.tensor(offs, device="cuda"), dev_status=status)
        good = fq.fp8_matmul_wgrad(a, sa, b, sb, torch.tensor(meant, device="cuda"))
        assert int(status) == 1 and torch.equal(out, good)


def test_same_bits_on_another_stream(fq):
    gen = torch.Generator(device="cuda").manual_seed(3)
    cap = fq.fp4_to_fp8_cols_scale_capacity(700, 1)
    a, b = codes((200, 700), gen), codes((264, 700), gen)
    sa, sb = torch.ones((cap, 200), device="cuda"), torch.ones((cap, 264), device="cuda")
    first = fq.fp8_matmul_wgrad(a, sa, b, sb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = fq.fp8_matmul_wgrad(a, sa, b, sb)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, other)


STARTS = [  # M, offsets of nine groups
    (1024, [0, 1, 16, 17, 145, 272, 400, 415, 900, 1023]),
    (1024, [0, 3, 131, 260, 388, 388, 401, 657, 658, 1024]),
    (1040, [0, 128, 256, 259, 264, 266, 300, 428, 1000, 1040]),
    (16, [0, 0, 0, 5, 5, 6, 15, 16, 16, 16]),
    (2048, [0, 134, 263, 392, 522, 680, 937, 1193, 1462, 2047]),
]


@pytest.mark.parametrize("M,starts", STARTS)
@pytest.mark.parametrize("N,K", [(1, 1), (130, 264), (500, 1020)])
def test_wgrad_of_groups_from_any_token(fq, M, starts, N, K):
    """Rows of M % 16 == 0 tokens, groups that start at any byte of them, tiles of
    one CTA and of a pair.  A group of NaN codes must not be seen in the others."""
    offs = np.array(starts)
    G = len(offs) - 1
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    cap = fq.fp4_to_fp8_cols_scale_capacity(M, G)
    a, sa = operands(M, N, offs, gen, cap)
    b, sb = operands(M, K, offs, gen, cap)
    dev = torch.from_numpy(offs).cuda()
    ref, mag, blocks = reference(a, sa, b, sb, offs)
    for dtype in (torch.float32, torch.bfloat16):
        out = fq.fp8_matmul_wgrad(a, sa, b, sb, dev, out_dtype=dtype)
        check(out, ref, mag, blocks)
        before = torch.randn((G, N, K), device="cuda", generator=gen).to(dtype)
        again = fq.fp8_matmul_wgrad(a, sa, b, sb, dev, out=before.clone(), accumulate=True)
        check(again, ref, mag, blocks, before)
    plain = fq.fp8_matmul_wgrad(a, sa, b, sb, dev)
    for g in (4, 7):
        x, y = a.clone(), b.clone()
        x[:, int(offs[g]):int(offs[g + 1])] = 0x7F
        y[:, int(offs[g]):int(offs[g + 1])] = 0xFF
        out = fq.fp8_matmul_wgrad(x, sa, y, sb, dev)
        keep = [i for i in range(G) if i != g]
        assert torch.equal(out[keep], plain[keep])
        assert bool(out[g].isnan().all()) == bool(offs[g + 1] > offs[g])
