"""GPU: the FP8 products on every dispatch path, with more tiles than the card
takes at once, so that the state carried from tile to tile (stages, accumulator
phases, scale slots, the next tile's first scales, the tile walk's refills) is
compared too.  Sizes are chosen for 152 SMs by the rules of launch_forward and
one_cta_tiles; on another count a case may take another path and is as valid.

The references and bounds are those of the products' other tests: the same
product in 64 bits, binary32 sums in any order."""
import numpy as np
import pytest
import torch

import test_gpu_matmul as dense
import test_gpu_wgrad as wgrad

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_quantization_gb300 as m
    m.abi()
    return m


def check_dense(fq, M, N, K, rows, dtype):
    y, ys, w, ws = dense.make(M, N, K, None, rows, M + N + K)
    out = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fq.fp8_matmul(y, ys, w, ws, out=out, dev_status=status)
    dense.check(out, dense.expand_rows(y, ys), dense.expand_weight(w, ws), K)
    assert int(status) == 0


@pytest.mark.parametrize("rows", [128, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [
    (3001, 5000, 640),    # pairs, 240 tiles on 76 clusters, output by tensor copies and rows
    (2999, 5003, 896),    # the same, rows of c not 16-byte aligned
    (2560, 4864, 128),    # pairs, one block a tile
    (2304, 2432, 1152),   # one CTA a tile, 342 tiles
    (20, 1000, 896),      # few rows (17 to 32), K split
    (32, 9000, 1152),     # few rows, K split in two
    (31, 50001, 384),     # few rows, 391 tiles on 304 CTAs
    (7, 60000, 640),      # few rows (up to 16), 469 tiles
])
def test_dense_paths(fq, M, N, K, rows, dtype):
    check_dense(fq, M, N, K, rows, dtype)


def test_dense_more_than_32_tiles_a_cluster(fq):
    check_dense(fq, 8200, 19000, 384, 128, torch.bfloat16)
    check_dense(fq, 8200, 19000, 256, 1, torch.bfloat16)


def spread(G, total, seed):
    """Counts of G groups, a fifth of them empty, that add up to total."""
    rng = np.random.default_rng(seed)
    p = rng.random(G) + 0.2
    p[rng.permutation(G)[:G // 5]] = 0
    return np.bincount(rng.choice(G, size=total, p=p / p.sum()), minlength=G)


@pytest.mark.parametrize("rows", [128, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,total,rest,N,K", [
    (6, 600, 0, 4104, 640),      # mean 100: one CTA a tile, 264 tiles and more
    (8, 400, 10, 1400, 896),     # mean 51, 88 and more columns of tiles: one CTA a tile
    (5, 640, 1, 1003, 384),      # mean 128 and a bit: pairs; rows of c not aligned
    (7, 5000, 3, 2056, 640),     # pairs, several tiles a cluster
    (40, 500, 5, 2056, 640),     # few rows (16), more than 680 tiles on 304 CTAs
    (20, 500, 0, 2600, 896),     # few rows (32), more than 420 tiles
    (3, 80, 2, 300, 1152),       # few rows (32), K split
    (2, 120, 0, 600, 1152),      # few rows (64), K split
    (300, 3000, 40, 200, 256),   # few rows (16), many groups
])
def test_ragged_paths(fq, G, total, rest, N, K, rows, dtype):
    counts = spread(G, total, G + N)
    M = total + rest
    offs = np.concatenate([[0], np.cumsum(counts)])
    y, ys, w, ws = dense.make(M, N, K, G, rows, G + K)
    out = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fq.fp8_matmul(y, ys, w, ws, torch.from_numpy(offs).cuda(), out=out, dev_status=status)
    for g in range(G):
        lo, hi = int(offs[g]), int(offs[g + 1])
        if hi > lo:
            dense.check(out[lo:hi], dense.expand_rows(y[lo:hi], ys[lo:hi]),
                        dense.expand_weight(w[g], ws[g]), K)
    assert bool((out[total:] == 0).all()) and int(status) == 0


@pytest.mark.parametrize("rows", [128, 1])
def test_ragged_more_than_32_tiles_a_cta(fq, rows):
    """Mean 100 rows, 40 groups and 123 columns of tiles: more than 4920 tiles of one
    CTA.  All of the rows in one group of 200 as well: 16-row tiles of that group."""
    test_ragged_paths(fq, 40, 4000, 0, 15700, 256, rows, torch.bfloat16)
    G, M, N, K = 200, 3000, 1032, 384
    y, ys, w, ws = dense.make(M, N, K, G, rows, 9)
    offs = torch.zeros(G + 1, dtype=torch.int64, device="cuda")
    offs[78:] = M
    out = fq.fp8_matmul(y, ys, w, ws, offs)
    dense.check(out, dense.expand_rows(y, ys), dense.expand_weight(w[77], ws[77]), K)


def check_wgrad(fq, a, sa, b, sb, offs, dev, gen):
    ref, mag, blocks = wgrad.reference(a, sa, b, sb, offs)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        out = fq.fp8_matmul_wgrad(a, sa, b, sb, dev, out_dtype=dtype, dev_status=status)
        wgrad.check(out, ref, mag, blocks)
        before = torch.randn(out.shape, device="cuda", generator=gen).to(dtype)
        again = fq.fp8_matmul_wgrad(a, sa, b, sb, dev, out=before.clone(), accumulate=True,
                                    dev_status=status)
        wgrad.check(again, ref, mag, blocks, before)
    assert int(status) == 0


@pytest.mark.parametrize("G,M,rest,N,K", [
    (6, 2000, 0, 1300, 1500),    # pairs, 216 tiles on 76 clusters, some groups empty
    (6, 1999, 8, 1301, 1502),    # the same, rows of c not 16-byte aligned
    (40, 3000, 0, 520, 1000),    # one CTA a tile, 1600 tiles
    (3, 900, 1, 700, 900),       # one CTA a tile
    (72, 5000, 0, 1500, 1500),   # pairs, more than 32 tiles a cluster
])
def test_wgrad_paths(fq, G, M, rest, N, K):
    counts = spread(G, M, G + N)
    offs = np.concatenate([[0], np.cumsum(counts)])
    gen = torch.Generator(device="cuda").manual_seed(G + K)
    cap = fq.fp4_to_fp8_cols_scale_capacity(M + rest, G)
    a, sa = wgrad.operands(M + rest, N, offs, gen, cap)
    b, sb = wgrad.operands(M + rest, K, offs, gen, cap)
    check_wgrad(fq, a, sa, b, sb, offs, torch.from_numpy(offs).cuda(), gen)


@pytest.mark.parametrize("M", [1008, 1001])
@pytest.mark.parametrize("N,K", [(4090, 4860), (2100, 2300)])
def test_wgrad_of_one_group_paths(fq, M, N, K):
    """In place (M % 16 == 0) and re-laid; pairs with four tiles a cluster, one CTA."""
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    offs, cap = np.array([0, M]), fq.fp4_to_fp8_cols_scale_capacity(M, 1)
    a, sa = wgrad.operands(M, N, offs, gen, cap)
    b, sb = wgrad.operands(M, K, offs, gen, cap)
    check_wgrad(fq, a, sa, b, sb, offs, None, gen)
