"""int8_linear's form that casts its tokens in the product's launch (GPU): rows of codes that end
inside one of its ranges of K, against the 64-bit definition (oracle/block.py).

The sums are exact, so the tolerances are test_gpu_int8's: the conversion of the sum, two products and one
sum in binary32, then the output's type."""
import numpy as np
import pytest
import torch

import oracle.block as OB
import scaled_quantization_amd as sq
from gpu_util import DEV
from test_gpu_block_norm import IDS, TYPES, draw, f64
from test_gpu_int8 import check_product, codes_of

pytestmark = pytest.mark.gpu


def linear(x, w8, w_scale, bias=None):
    y = torch.full((x.shape[0], w8.shape[0]), float("nan"), dtype=x.dtype, device=DEV)
    ws = torch.empty(sq.int8_linear_workspace(*x.shape), dtype=torch.uint8, device=DEV)
    sq.int8_linear(x.to(DEV), w8, w_scale, y, ws, bias)
    return y


def check_linear(x, w8, w_scale, what):
    q, s = OB.quantize_int8(f64(x))
    check_product(linear(x, w8, w_scale), q, w8.cpu().numpy(), s.astype(np.float32),
                  f64(w_scale).astype(np.float32), None, x.dtype, what)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 16])
@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_every_length_of_short_rows(t, M):
    # A piece of K is 128 codes: those behind a shorter row must be zeros, whichever range of the row a
    # wave casts.  A call with codes of 127 throughout leaves such codes in every compute unit's LDS first.
    many = torch.ones((2, 4096), dtype=t)
    many_w8, many_scale = codes_of(torch.ones((4096, 4096), dtype=t))
    for K in range(16, 16384 // max(M, 16) + 1, 16):
        w8, w_scale = codes_of(draw((40, K), t, K, 0.02))
        linear(many, many_w8, many_scale)
        check_linear(draw((M, K), t, K + 1), w8, w_scale, f"{M} tokens, K {K}")


@pytest.mark.parametrize("t, M, K", [
    # the longest rows that are cast in the product's launch, and the next ones, which are not
    (torch.bfloat16, 1, 20480), (torch.bfloat16, 1, 20496), (torch.float16, 1, 20480), (torch.float16, 1, 20496),
    (torch.float32, 1, 12288), (torch.float32, 1, 12304), (torch.bfloat16, 4, 4096), (torch.bfloat16, 4, 4112),
    (torch.float16, 16, 1024), (torch.float16, 16, 1040), (torch.float32, 16, 768), (torch.float32, 16, 784),
    (torch.float32, 7, 1744), (torch.float32, 7, 1760)])
def test_longest_rows_that_are_cast_in_the_launch(t, M, K):
    w8, w_scale = codes_of(draw((100, K), t, 2, 0.02))
    check_linear(draw((M, K), t, 1), w8, w_scale, f"{M} tokens, K {K}")
