"""Counts that do not fit the C ABI's 32-bit arguments are refused by the binding
instead of being cut to their low 32 bits.  No call here reaches the library's
launches."""
import pytest
import torch


@pytest.fixture(scope="module")
def fq():
    from fp8_quantization_gb300 import build
    build.build()
    import fp8_quantization_gb300 as m
    m.abi()
    return m


WRAPS = [2 ** 32 + 2, -2 ** 32 + 2, 2 ** 31]


@pytest.mark.parametrize("v", WRAPS)
def test_route_refuses_counts_past_32_bits(fq, v):
    logits = torch.zeros((0, 16))
    for name in ("n_groups", "keep_groups", "group_top"):
        with pytest.raises(ValueError, match=name):
            fq.moe_route(logits, 2, **{"n_groups": 2, name: v})
    with pytest.raises(ValueError, match="k must"):
        fq.moe_route(logits, v)


@pytest.mark.parametrize("v", WRAPS)
def test_sort_refuses_counts_past_32_bits(fq, v):
    with pytest.raises(ValueError, match="n_experts"):
        fq.moe_sort_rows(torch.zeros(4, dtype=torch.int32), v)


@pytest.mark.parametrize("v", WRAPS)
def test_workspace_sizes_of_counts_past_32_bits(fq, v):
    assert fq.moe_sort_rows_workspace(9000, v) == -1
    assert fq.fp8_matmul_wgrad_workspace(100, 8, 8, v) == -1
