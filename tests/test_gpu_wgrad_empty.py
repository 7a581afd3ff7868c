"""GPU: the weight gradient of an empty batch through the C ABI, without group
offsets and, as the header allows there, without operands or a workspace."""
import ctypes

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


@pytest.mark.parametrize("N,K", [(1, 1), (40, 264), (300, 520), (4864, 4096)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("accumulate", [0, 1])
def test_no_tokens_need_no_workspace(fq, N, K, dtype, accumulate):
    c = torch.full((N, K), 3.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    cap = fq.fp4_to_fp8_cols_scale_capacity(0, 1)
    rc = fq.abi().fp8_matmul_wgrad(None, None, N, None, None, K, 0, None, 1, cap,
                                   ctypes.c_void_p(c.data_ptr()), int(dtype == torch.float32),
                                   accumulate, None, 0, ctypes.c_void_p(status.data_ptr()),
                                   ctypes.c_void_p(stream))
    assert rc == 0
    assert bool((c == (3.0 if accumulate else 0.0)).all()) and int(status) == 0


@pytest.mark.parametrize("offsets", [None, [0, 0], [0, 0, 0, 0]])
def test_no_tokens_through_the_binding(fq, offsets):
    G = 1 if offsets is None else len(offsets) - 1
    dev = None if offsets is None else torch.tensor(offsets, device="cuda")
    cap = fq.fp4_to_fp8_cols_scale_capacity(0, G)
    a, b = (torch.empty((n, 0), dtype=torch.uint8, device="cuda") for n in (72, 136))
    sa, sb = (torch.full((cap, n), float("nan"), device="cuda") for n in (72, 136))
    assert bool((fq.fp8_matmul_wgrad(a, sa, b, sb, dev) == 0).all())
    out = torch.full((G, 72, 136), 5.0, device="cuda")
    fq.fp8_matmul_wgrad(a, sa, b, sb, dev, out=out, accumulate=True)
    assert bool((out == 5).all())
