"""Sizes next to the end of an int, without a GPU: the products' tiling rounds sizes up to whole tiles
in int arithmetic, so what it cannot round up is refused before any of it runs."""
import ctypes

import pytest

import gemv_w4a16_w8a8_b200 as qg

P = [ctypes.c_void_p(0x100000 * i) for i in range(1, 11)]      # never dereferenced
MOST = 2 ** 31 - 4096                                          # rows or columns
BEYOND = [MOST + 1, 2 ** 31 - 256, 2 ** 31 - 255, 2 ** 31 - 1]


def scaled(M=4, N=64, K=64):
    return qg.lib().qgemm_w8a8_scaled(*P[:4], None, P[4], M, N, K, 0, None)


def gated8(M=4, N=64, K=64):
    return qg.lib().qgemm_w8a8_gated(*P[:7], M, N, K, 0, 0, None)


def gated(M=4, N=64, K=64):
    return qg.lib().qgemm_dense_gated(*P[:4], None, None, M, N, K, 0, 0, None)


def backward(M=4, N=64, K=64):
    return qg.lib().qgemm_dense_gated_backward(*P[:9], M, N, K, 0, 0, P[9], 2 ** 64 - 1, None)


@pytest.mark.parametrize("call", [scaled, gated8, gated, backward])
@pytest.mark.parametrize("which", ["M", "N"])
@pytest.mark.parametrize("size", BEYOND)
def test_too_many_rows_or_columns(call, which, size):
    assert call(**{which: size}) == qg.QG_ERR_UNSUPPORTED_SHAPE


@pytest.mark.parametrize("call", [gated, backward])
@pytest.mark.parametrize("size", [MOST + 8, 2 ** 31 - 8])
def test_too_long_a_reduction(call, size):
    assert call(K=size) == qg.QG_ERR_UNSUPPORTED_SHAPE


def test_no_workspace_for_sizes_that_are_refused():
    size = qg.qgemm_dense_gated_backward_workspace_bytes
    for n in BEYOND:
        assert size(n, 8, 8) == size(8, n, 8) == 0
    assert size(8, 8, 2 ** 31 - 8) == 0
    # the largest that is taken: dG and dU alone, rows of eight values
    assert size(MOST, 1, 8) >= 2 * MOST * 16
    assert size(MOST, MOST, 8) >= 4 * MOST * MOST
