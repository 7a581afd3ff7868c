"""GPU: group_sum_rows of long groups, whose pieces are added up by a second kernel, at the
edges of pieces of 128, 256 and 512 rows.  Small integers: every partial sum is exact in
binary32 (at most 4 * 299500 < 2^24), so that a row left out or taken twice shows."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]
EDGES = [511, 512, 513, 0, 1, 1024, 1025, 127, 128, 129, 255, 256, 257, 4096, 3, 4097]


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_quantization_gb300 as m
    m.abi()
    return m


def integers(shape, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-4, 5, shape, device="cuda", generator=gen, dtype=torch.int8).to(dtype)


def sums(x, bounds):
    """In 64 bits, some rows at a time."""
    out = torch.zeros((len(bounds) - 1, x.shape[1]), dtype=torch.float64, device="cuda")
    for g, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        for at in range(lo, hi, 16384):
            out[g] += x[at:min(at + 16384, hi)].double().sum(0)
    return out


# rows of the longest group: pieces of 128 rows up to 16384 rows in all, of 256 or, where
# there are columns enough, of 512
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("longest,N", [(1000, 520), (1000, 2049), (9001, 520), (9001, 1001), (8200, 4096),
                                       (8191, 4100), (30001, 2056), (30001, 2049), (150000, 600)])
def test_edges_of_pieces(fq, longest, N, dtype):
    counts = EDGES + [longest] + EDGES[::-1] * (longest > 8000)
    bounds = [0] + torch.tensor(counts).cumsum(0).tolist()
    M = bounds[-1] + 77  # 77 rows of no group
    x = integers((M, N), dtype, M + N)
    x[bounds[-1]:] = float("nan")
    offs = torch.tensor(bounds, device="cuda")
    want = sums(x, bounds)
    out = fq.group_sum_rows(x, offs, out=torch.full(want.shape, float("nan"), device="cuda"))
    assert torch.equal(out.double(), want)
    more = fq.group_sum_rows(x, offs, out=(100 * want).float(), accumulate=True)
    assert torch.equal(more.double(), 101 * want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N", [(2049, 8), (16384, 1000), (16385, 1000), (20011, 7168), (100003, 2056), (100003, 300)])
def test_one_group(fq, M, N, dtype):
    x = integers((M, N), dtype, M)
    assert torch.equal(fq.group_sum_rows(x).double(), sums(x, [0, M]))


def test_rows_past_32_bit_offsets(fq):
    """300000 rows of 7168 BF16: 2.15 G elements, both groups of many pieces."""
    M, N = 300000, 7168
    x = integers((M, N), torch.bfloat16, 1)
    bounds = [0, 299500 - 1030, M]
    out = fq.group_sum_rows(x, torch.tensor(bounds, device="cuda"))
    assert torch.equal(out.double(), sums(x, bounds))
