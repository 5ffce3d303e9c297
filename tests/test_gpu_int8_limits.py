"""INT8 products whose workgroups have more threads in all than one launch takes (GPU).

The sums are exact and the epilogue is (sum sa) sb, a binary32 rounding each, then y's type: the same steps
on a tensor of the sums give the same values."""
import pytest
import torch

import scaled_quantization_amd as sq
from gpu_util import DEV

pytestmark = pytest.mark.gpu

N_WIDE = (1 << 27) + 100        # 16 channels a workgroup of 512 threads: past 2^32 threads


def codes(*shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-128, 128, shape, dtype=torch.int8, generator=g, device=DEV)


def floats(n, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.rand(n, generator=g, device=DEV) * 0.02 + 0.001


def same(y, sums, sa, sb, what):
    """y [M, n] against the epilogue's steps on integer sums held as float32."""
    want = ((sums * sa[:, None]) * sb).to(y.dtype)
    assert torch.equal(y, want), f"{what}: {int((y != want).sum())} of {y.numel()} differ"


@pytest.mark.parametrize("M, K", [(1, 1), (2, 16), (50, 3)])
def test_int8_gemm_of_few_tokens_and_very_many_channels(M, K):
    a, b, sa, sb = codes(M, K, seed=1), codes(N_WIDE, K, seed=2), floats(M, 3), floats(N_WIDE, 4)
    y = torch.full((M, N_WIDE), float("nan"), dtype=torch.bfloat16, device=DEV)
    sq.int8_gemm(a, b, sa, sb, y)
    for n in range(0, N_WIDE, 1 << 24):
        part = slice(n, n + (1 << 24))
        sums = torch.zeros((M, b[part].shape[0]), device=DEV)
        for k in range(K):
            sums += a[:, k].float()[:, None] * b[part, k].float()
        same(y[:, part], sums, sa, sb[part], f"channels from {n}")


def test_int8_linear_of_one_token_and_very_many_channels():
    K = 16                       # cast in the product's launch
    x = torch.linspace(-3, 3, K, device=DEV).bfloat16()[None, :]
    b, sb = codes(N_WIDE, K, seed=2), floats(N_WIDE, 4)
    q, sa = torch.empty((1, K), dtype=torch.int8, device=DEV), torch.empty(1, device=DEV)
    sq.quantize_int8(x, q, sa)
    y = torch.full((1, N_WIDE), float("nan"), dtype=torch.bfloat16, device=DEV)
    sq.int8_linear(x, b, sb, y, torch.empty(sq.int8_linear_workspace(1, K), dtype=torch.uint8, device=DEV))
    for n in range(0, N_WIDE, 1 << 24):
        part = slice(n, n + (1 << 24))
        same(y[:, part], (b[part].float() * q.float()).sum(1)[None, :], sa, sb[part], f"channels from {n}")


@pytest.mark.parametrize("M, N, K", [(1 << 30, 1, 1), ((1 << 24) + 77, 2049, 1)])
def test_int8_gemm_of_very_many_tiles(M, N, K):
    # rows below 16 bytes: tiles of 64 x 64, 2^24 and more of them
    a, b, sa, sb = codes(M, K, seed=1), codes(N, K, seed=2), floats(M, 3), floats(N, 4)
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    sq.int8_gemm(a, b, sa, sb, y)
    step = (1 << 26) // N
    for m in range(0, M, step):
        part = slice(m, m + step)
        same(y[part], a[part].float() * b.float().T, sa[part], sb, f"rows from {m}")
