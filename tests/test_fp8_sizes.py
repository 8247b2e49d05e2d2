"""Sizes next to 2^31, whose rounding up to tiles and grids does not fit 32 bits, are refused before any launch (CPU)."""
import ctypes

import pytest

import bit_quantized_gemm_group_b200 as q

A = ctypes.c_void_p(0x10000)    # never dereferenced: validation fails first
WS = (A, 1 << 62)
TOP = 2 ** 31
SHAPE, NULL = 2, 1


def gemm(M=4, K=256, N=64, Y=A):
    return q.lib().qg_gemm_fp8(A, A, M, K, A, A, N, Y, 1, *WS, None)


def experts(S=8, K=256, N=64, token=A, Y=A):
    return q.lib().qg_gemm_fp8_experts(A, A, TOP - 1, K, token, A, S, 4, A, A, N, Y, 1, *WS, None)


@pytest.mark.parametrize("call", [gemm, experts])
@pytest.mark.parametrize("name", ["K", "N"])
def test_products_k_and_n(call, name):
    assert call(**{name: TOP - 16}) == call(**{name: TOP - 240}) == SHAPE
    assert call(**{name: TOP - 256}, Y=None) == (SHAPE if (call, name) == (experts, "K") else NULL)


@pytest.mark.parametrize("call,name", [(gemm, "M"), (experts, "S")])
def test_products_rows(call, name):
    assert call(**{name: TOP - 1}) == call(**{name: TOP - 255}) == SHAPE
    assert call(**{name: TOP - 256}, Y=None) == NULL


def test_experts_rows_by_a_map_have_a_grid():
    assert experts(K=65535 * 4096 + 16) == SHAPE
    assert experts(K=65535 * 4096, Y=None) == NULL
    assert q.lib().qg_gemm_fp8_experts(A, A, 8, 65535 * 4096 + 16, None, A, 8, 4, A, A, 64, None, 1, *WS, None) == NULL


def test_workspace_of_refused_sizes_is_none():
    for op in (q.QG_OP_GEMM_FP8, q.QG_OP_GEMM_FP8_EXPERTS):
        for M, K, N in ((TOP - 1, 256, 64), (4, TOP - 16, 64), (4, 256, TOP - 16)):
            assert q.qg_workspace_size(op, M, K, N) == 0
        assert q.qg_workspace_size(op, TOP - 256, 8192, 64) > 0


def test_weight_quantizer():
    f = q.lib().qg_quantize_weight_fp8
    assert f(A, 2, 1, TOP - 16, 64, A, A, None) == f(A, 2, 1, 256, TOP - 16, A, A, None) == SHAPE


def test_router():
    def route(M, idx):
        return q.lib().qg_route_topk(A, 2, M, 64, None, 0, 1, 1, 1, 8, 1, ctypes.c_float(1.0), idx, A, None)
    assert route(TOP - 1, A) == route(TOP - 3, A) == SHAPE
    assert route(TOP - 4, None) == NULL
