"""Refusals of the block norm and its gradient that tests/test_gated_host.py does not hold (C ABI, no GPU is reached)."""
import os

import pytest

import scaled_quantization_amd as sq


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(sq.LIB_PATH):
        pytest.skip("libfp8dp.so not built")
    return sq.lib()


def refused(L, rc, word):
    assert rc == -1 and word in L.fp8dp_last_error(), (rc, L.fp8dp_last_error())


# addresses that are never read: every call below is refused
def norm(L, x=16, res=32, post=48, gate=64, tok=0, pre=80, dt=0, gt=0, z=96, y=112, r1=128, r2=144):
    return L.block_norm(x, res, post, gate, tok, pre, 4, 8, dt, dt, gt, 1.0, 1.0, 1e-5, z, y, r1, r2, None)


def test_statistics_of_a_norm_that_is_not_there(L):
    # they would stay as they were
    refused(L, norm(L, y=None), b"pre_rstd belongs to y")
    refused(L, norm(L, y=None, pre=None), b"pre_rstd belongs to y")
