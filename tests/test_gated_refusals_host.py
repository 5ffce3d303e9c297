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


def test_norm_outputs_that_are_one_buffer_or_an_input(L):
    # (y over z, x and residual: tests/test_gated_host.py)
    for kw in ({"y": 48}, {"y": 80}, {"y": 64}, {"y": 64, "tok": 1}, {"y": 128}, {"y": 144},
               {"z": 48}, {"z": 80}, {"z": 64}, {"z": 128}, {"z": 144},
               {"r1": 144}, {"r1": 16}, {"r2": 32}, {"r1": 48}, {"r2": 64}, {"r2": 80}):
        refused(L, norm(L, **kw), b"must not be")


def backward(L, dy=16, add=32, x=48, z=64, post=80, gate=96, tok=0, pre=112, r1=128, r2=144, dres=160, dx=176, dgate=192,
             dpost=208, dpre=224, ws=240):
    return L.block_norm_backward(dy, add, x, z, post, gate, tok, pre, r1, r2, 4, 8, 2, 2, 2, 1.0, 1.0, dres, dx, dgate,
                                 dpost, dpre, ws, None)


def test_gradients_that_are_one_buffer_or_an_input(L):
    outs = {"dres": 160, "dx": 176, "dgate": 192, "dpost": 208, "dpre": 224}
    ins = {"x": 48, "z": 64, "post": 80, "gate": 96, "pre": 112, "r1": 128, "r2": 144, "ws": 240}
    for tok in (0, 1):
        for out in outs:
            for where in [v for k, v in outs.items() if k != out] + list(ins.values()):
                refused(L, backward(L, tok=tok, **{out: where}), b"different buffers")
    # in place of dy and dz_add are the gradients of the activations' shape alone
    for out in ("dpost", "dpre", "dgate"):
        for where in (16, 32):
            refused(L, backward(L, **{out: where}), b"different buffers")
