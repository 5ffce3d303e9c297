"""Limits of the INT8 product that are refused before anything is launched.  No call here reaches a GPU."""
import os

import pytest

import scaled_quantization_amd as sq


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(sq.LIB_PATH):
        pytest.skip("libfp8dp.so not built")
    return sq.lib()


@pytest.mark.parametrize("M, N", [(1 << 30, (1 << 10) + 1), ((1 << 10) + 1, 1 << 30), (1 << 30, 1 << 30)])
@pytest.mark.parametrize("K", [1, 16, 17, 4096, sq.INT8_MAX_K])
def test_more_outputs_than_indexes(L, M, N, K):
    # refused as a whole, also by the call that would cast its tokens first
    rc = L.int8_gemm(16, 16, M, N, K, 16, 16, None, 0, 0, 16, None, 0, None)
    assert rc == -1 and b"2^40" in L.fp8dp_last_error(), L.fp8dp_last_error()
    rc = L.int8_linear(16, 16, 16, None, M, N, K, 0, 0, 16, 16, L.int8_linear_workspace(M, K), None)
    assert rc == -1 and b"2^40" in L.fp8dp_last_error(), L.fp8dp_last_error()
