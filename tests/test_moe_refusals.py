"""The mixture-of-experts and FP8 product calls refuse bad arguments: the C ABI on
the host before anything is enqueued, the binding before the ABI.  No call here
reaches a CUDA API."""
import ctypes

import pytest
import torch

OK, NULL, SHAPE, ALIGN, ARG = 0, 1, 2, 3, 4
P = ctypes.c_void_p(0x1000)   # 16-byte aligned fake device pointer (never dereferenced)
PM = ctypes.c_void_p(0x1008)  # misaligned


@pytest.fixture(scope="module")
def fq():
    from fp8_quantization_gb300 import build
    build.build()
    import fp8_quantization_gb300 as m
    m.abi()
    return m


def test_abi_matmul(fq):
    f = fq.abi().fp8_matmul
    # a, sa, M, K, b, sb, N, b_block, offsets, G, c, c_f32, status, stream
    assert f(P, P, -1, 128, P, P, 64, 128, None, 1, P, 0, None, None) == SHAPE
    assert f(P, P, 4, 96, P, P, 64, 128, None, 1, P, 0, None, None) == SHAPE
    assert f(P, P, 4, 0, P, P, 64, 128, None, 1, P, 0, None, None) == SHAPE
    assert f(P, P, 4, 128, P, P, 0, 128, None, 1, P, 0, None, None) == SHAPE
    assert f(P, P, 2 ** 31, 128, P, P, 64, 128, None, 1, P, 0, None, None) == SHAPE
    assert f(P, P, 4, 128, P, P, 2 ** 30, 128, P, 4, P, 0, None, None) == SHAPE
    assert f(P, P, 4, 128, P, P, 64, 64, None, 1, P, 0, None, None) == ARG
    assert f(P, P, 4, 128, P, P, 64, 128, None, 2, P, 0, None, None) == ARG    # no offsets, G = 2
    assert f(P, P, 4, 128, P, P, 64, 128, P, 0, P, 0, None, None) == ARG
    assert f(P, P, 4, 128, P, P, 64, 128, P, 1025, P, 0, None, None) == ARG
    assert f(P, P, 4, 128, P, P, 64, 128, None, 1, P, 2, None, None) == ARG
    assert f(P, P, 4, 128, P, P, 64, 128, None, 1, None, 0, None, None) == NULL
    assert f(P, None, 4, 128, P, P, 64, 128, None, 1, P, 0, None, None) == NULL
    assert f(P, P, 4, 128, PM, P, 64, 128, None, 1, P, 0, None, None) == ALIGN
    assert f(P, P, 4, 128, P, P, 64, 128, PM, 1, P, 0, None, None) == ALIGN
    assert f(None, None, 0, 128, None, None, 64, 128, None, 1, None, 0, None, None) == OK


def test_abi_cols_and_wgrad(fq):
    c = fq.abi().fp8_quantize_cols
    # x, M, K, offsets, G, yT, scale, cap, status, stream
    assert c(P, 100, 12, P, 4, P, P, 5, None, None) == SHAPE
    assert c(P, -1, 64, P, 4, P, P, 5, None, None) == SHAPE
    assert c(P, 100, 64, P, 0, P, P, 5, None, None) == ARG
    assert c(P, 100, 64, None, 2, P, P, 5, None, None) == ARG
    assert c(P, 100, 64, P, 4, P, P, 4, None, None) == ARG       # cap too small
    assert c(P, 100, 64, P, 4, None, P, 5, None, None) == NULL
    assert c(PM, 100, 64, P, 4, P, P, 5, None, None) == ALIGN
    n = fq.abi().fp8_matmul_wgrad_workspace
    assert n(100, 3, 5, 4) == 8 * 128 * 5 and n(0, 1, 1, 1) == 256
    assert n(-1, 3, 5, 4) == -1 and n(100, 0, 5, 4) == -1 and n(100, 3, 5, 0) == -1
    assert n(2 ** 31 - 600, 3, 5, 4) == -1
    f = fq.abi().fp8_matmul_wgrad
    # aT, sa, N, bT, sb, K, M, offsets, G, cap, c, f32, add, ws, ws_bytes, status, stream
    W = 8 * 128 * 5
    assert f(P, P, 3, P, P, 5, 100, P, 4, 5, P, 1, 0, P, W - 1, None, None) == ARG
    assert f(P, P, 3, P, P, 5, 100, P, 4, 4, P, 1, 0, P, W, None, None) == ARG
    assert f(P, P, 3, P, P, 5, 100, P, 4, 5, P, 1, 2, P, W, None, None) == ARG
    assert f(P, P, 3, P, P, 5, 100, None, 4, 5, P, 1, 0, P, W, None, None) == ARG
    assert f(P, P, 0, P, P, 5, 100, P, 4, 5, P, 1, 0, P, W, None, None) == SHAPE
    assert f(P, P, 2 ** 30, P, P, 5, 100, P, 4, 5, P, 1, 0, P, 2 ** 62, None, None) == SHAPE
    assert f(P, P, 3, None, P, 5, 100, P, 4, 5, P, 1, 0, P, W, None, None) == NULL
    assert f(P, P, 3, P, P, 5, 100, P, 4, 5, P, 1, 0, None, W, None, None) == NULL
    assert f(P, P, 3, P, P, 5, 100, P, 4, 5, P, 1, 0, PM, W, None, None) == ALIGN


def test_abi_route_and_sort(fq):
    f = fq.abi().moe_route
    # logits, f32, T, E, k, bias, sigmoid, n_groups, keep, top, renorm, scale, w, ids, stream
    good = [P, 1, 4, 64, 8, None, 0, 8, 4, 2, 1, 1.0, P, P, None]

    def bad(i, v, code):
        args = list(good)
        args[i] = v
        assert f(*args) == code, (i, v)

    for i, v in ((1, 2), (3, 0), (3, 1025), (4, 0), (4, 65), (4, 33), (6, 3), (7, 0), (7, 7), (7, 64),
                 (8, 0), (8, 9), (9, 0), (9, 3), (10, 2)):
        bad(i, v, ARG)
    bad(2, -1, SHAPE)
    bad(0, None, NULL)
    bad(12, None, NULL)
    bad(13, PM, ALIGN)
    bad(5, PM, ALIGN)
    bad(2, 0, OK)
    b = fq.abi().moe_route_backward
    # logits, f32, T, E, ids, dw, k, sigmoid, renorm, scale, dlogits, stream
    assert b(P, 1, -1, 64, P, P, 8, 0, 1, 1.0, P, None) == SHAPE
    assert b(P, 1, 4, 64, P, P, 65, 0, 1, 1.0, P, None) == ARG
    assert b(P, 1, 4, 64, None, P, 8, 0, 1, 1.0, P, None) == NULL
    assert b(P, 1, 4, 64, P, P, 8, 0, 1, 1.0, PM, None) == ALIGN
    assert b(None, 1, 0, 64, None, None, 8, 0, 1, 1.0, None, None) == OK
    w = fq.abi().moe_sort_rows_workspace
    assert w(0, 4) == 0 and w(8192, 1024) == 0 and w(8193, 16) == 3 * 16 * 4
    assert w(-1, 4) == -1 and w(10, 0) == -1 and w(10, 1025) == -1
    s = fq.abi().moe_sort_rows
    # ids, n, E, offsets, pair, row, ws, ws_bytes, stream
    assert s(P, -1, 4, P, P, P, None, 0, None) == SHAPE
    assert s(P, 10, 0, P, P, P, None, 0, None) == ARG
    assert s(P, 9000, 4, P, P, P, P, 10, None) == ARG
    assert s(P, 10, 4, None, P, P, None, 0, None) == NULL
    assert s(P, 10, 4, P, PM, P, None, 0, None) == ALIGN


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def f32(*shape):
    return torch.zeros(shape, dtype=torch.float32)


def raises(fn, match):
    with pytest.raises(ValueError, match=match):
        fn()


def test_binding_matmul(fq):
    y, ys, w, ws = u8(4, 256), f32(4, 2), u8(200, 256), f32(2, 2)
    offs = torch.tensor([0, 4])
    raises(lambda: fq.fp8_matmul(y.float(), ys, w, ws), "uint8")
    raises(lambda: fq.fp8_matmul(y, f32(4, 3), w, ws), "ys must have shape")
    raises(lambda: fq.fp8_matmul(y, ys, u8(200, 128), ws), "w must have shape")
    raises(lambda: fq.fp8_matmul(y, ys, w, f32(3, 2)), "ws must have shape")
    raises(lambda: fq.fp8_matmul(y, ys, w, ws, offs), "3 dimensions")
    raises(lambda: fq.fp8_matmul(y, ys, w[None], ws[None], torch.tensor([0, 2, 4])), "w must have shape")
    raises(lambda: fq.fp8_matmul(y, ys, w, ws, out_dtype=torch.float16), "bfloat16 or float32")
    raises(lambda: fq.fp8_matmul(y, ys, w, ws, out=f32(4, 199)), "out must have")
    raises(lambda: fq.fp8_matmul(u8(8, 256)[::2], ys, w, ws), "contiguous")
    raises(lambda: fq.fp8_matmul(y, ys, w, ws, dev_status=torch.zeros(0, dtype=torch.int32)), "dev_status")
    raises(lambda: fq.fp8_matmul(y, ys, w, ws), "CUDA tensor")


def test_binding_cols_and_wgrad(fq):
    x = torch.zeros((300, 64), dtype=torch.bfloat16)
    offs = torch.tensor([0, 100, 300])
    raises(lambda: fq.fp8_quantize_cols(x.float(), offs), "bfloat16")
    raises(lambda: fq.fp8_quantize_cols(x, offs.int()), "int64")
    raises(lambda: fq.fp8_quantize_cols(x, offs, yT=u8(64, 299)), "yT must have")
    raises(lambda: fq.fp8_quantize_cols(x, offs, yT_scale=f32(4, 64)), "yT_scale must be")
    raises(lambda: fq.fp8_quantize_cols(x, offs), "CUDA tensor")
    a, sa, b, sb = u8(64, 300), f32(5, 64), u8(128, 300), f32(5, 128)
    raises(lambda: fq.fp8_matmul_wgrad(a, sa, u8(128, 299), sb, offs), "tokens")
    raises(lambda: fq.fp8_matmul_wgrad(a, f32(4, 64), b, sb, offs), "aT_scale must be")
    raises(lambda: fq.fp8_matmul_wgrad(a, sa, b, f32(5, 127), offs), "bT_scale must be")
    raises(lambda: fq.fp8_matmul_wgrad(a, sa, b, sb, offs, out=f32(2, 64, 127)), "out must have")
    raises(lambda: fq.fp8_matmul_wgrad(a, sa, b, sb, offs, accumulate=True), "accumulate needs out")
    raises(lambda: fq.fp8_matmul_wgrad(a, sa, b, sb, offs, workspace=u8(10)), "workspace must hold")
    raises(lambda: fq.fp8_matmul_wgrad(a, sa, b, sb, offs), "CUDA tensor")


def test_binding_route_and_sort(fq):
    l = f32(4, 16)
    raises(lambda: fq.moe_route(l, 2, score="relu"), "softmax")
    raises(lambda: fq.moe_route(l.double(), 2), "float32 or bfloat16")
    raises(lambda: fq.moe_route(l, 2, bias=f32(15)), "bias must have")
    raises(lambda: fq.moe_route(l, 2, weights=f32(4, 3)), "weights must have")
    raises(lambda: fq.moe_route(l, 2, ids=f32(4, 2)), "int32")
    raises(lambda: fq.moe_route(l, 2), "CUDA tensor")
    ids = torch.zeros((4, 2), dtype=torch.int32)
    raises(lambda: fq.moe_route_backward(l, ids.long(), f32(4, 2)), "int32")
    raises(lambda: fq.moe_route_backward(l, ids, f32(4, 3)), "dweights must have")
    raises(lambda: fq.moe_route_backward(l, ids[:3], f32(4, 2)), "ids must have")
    raises(lambda: fq.moe_route_backward(l, ids, f32(4, 2)), "CUDA tensor")
    raises(lambda: fq.moe_sort_rows(ids.long(), 4), "int32")
    raises(lambda: fq.moe_sort_rows(ids, 4, pair_of_row=torch.zeros(7, dtype=torch.int32)), "pair_of_row")
    raises(lambda: fq.moe_sort_rows(torch.zeros(9000, dtype=torch.int32), 4, workspace=u8(8)), "workspace")
    raises(lambda: fq.moe_sort_rows(ids, 4), "CUDA tensor")
