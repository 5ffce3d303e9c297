"""Where the operators around the MLP keep more than their outputs' own rounding (GPU): INT8 codes
behind a norm, weight gradients of rows far from zero.

U = 2^-24 is a binary32 rounding."""
import numpy as np
import pytest
import torch

import oracle.block as OB
import scaled_quantization_amd as sq
from gpu_util import DEV
from test_gpu_block_norm import IDS, TYPES, U, close, draw, f64

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ codes behind a norm
@pytest.mark.parametrize("cols", [5, 100, 768, 4099, 8200, 20000])
@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_codes_behind_a_norm_at_the_borders(t, cols):
    # weight 0 makes the norm's binary32 values the bias: values at, just below and just above every border
    # between two codes, of which one in some has a binary32 product by 127 on the wrong side
    x, res = draw((3, cols), t, 1), draw((3, cols), t, 2)
    g = torch.Generator().manual_seed(cols)
    q = torch.empty((3, cols), dtype=torch.int8, device=DEV)
    scale = torch.empty(3, device=DEV)
    for top in (1.0, 3.0, 0.7, 1e-3, 333.3, 1e30, 1e-30):
        k = 2 * torch.randint(-127, 127, (cols,), generator=g) + 1
        b = (k.double() * float(np.float32(top)) / 254.0).float()
        step = torch.randint(-2, 3, (cols,), generator=g).to(torch.int32)
        b = (b.view(torch.int32) + step).view(torch.float32)
        b[0] = top
        want, s = OB.quantize_int8(f64(b)[None, :])
        for r in (None, res):
            z = None if r is None else torch.empty_like(x, device=DEV)
            sq.layer_norm_quantize_int8(x.to(DEV), torch.zeros(cols, device=DEV), b.to(DEV), 1e-5, q, scale,
                                        None if r is None else r.to(DEV), z)
            got = q.cpu().numpy()
            assert (got == want).all(), f"{top}: {(got != want).sum()} of {got.size} codes differ"
            close(scale, np.repeat(s, 3), U * s, "scale")


@pytest.mark.parametrize("rows, cols", [(8192, 4096), (1700, 20000)])
def test_codes_behind_a_norm_are_those_of_its_values(rows, cols):
    # the norm's binary32 values come out of layer_norm on the same values in float32: the same arithmetic
    x, w, b = draw((rows, cols), torch.bfloat16, 1).to(DEV), draw(cols, torch.float32, 2, 0.1, 1.0).to(DEV), \
        draw(cols, torch.float32, 3, 0.1).to(DEV)
    q, scale = torch.empty((rows, cols), dtype=torch.int8, device=DEV), torch.empty(rows, device=DEV)
    sq.layer_norm_quantize_int8(x, w, b, 1e-5, q, scale)
    y = torch.empty((rows, cols), device=DEV)
    sq.layer_norm(x.float(), w, b, 1e-5, y)
    v = y.double()
    top = v.abs().amax(1, keepdim=True)
    want = torch.round(v * 127.0 / top).to(torch.int8)       # 127 v is exact in 64 bits
    assert torch.equal(q, want), f"{int((q != want).sum())} of {q.numel()} codes differ"


# ------------------------------------------------------------------ gradients of rows far from zero
@pytest.mark.parametrize("cols", [7, 64, 768, 1001, 2048, 4096, 8192, 10000])
@pytest.mark.parametrize("t, mean", [(torch.bfloat16, 40.0), (torch.float16, 340.0), (torch.float32, 5000.0)],
                         ids=IDS)
def test_weight_gradient_of_rows_with_a_distant_mean(t, mean, cols):
    # h = (z - mean) rstd takes two roundings wherever the mean is; with the product's by dy and at
    # most rows - 1 of the sum a column is off by (rows + 3) U of its terms' magnitudes, one more for second order
    rows = 3
    z, dy = draw((rows, cols), t, cols, 1.0, mean), draw((rows, cols), t, 2)
    m = z.float().mean(1)
    r = 1.0 / torch.sqrt(z.float().var(1, unbiased=False) + 1e-5)
    dz, dw, db = torch.empty_like(z, device=DEV), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    ws = torch.empty(2 * rows * cols, device=DEV)
    sq.layer_norm_backward(dy.to(DEV), z.to(DEV), None, m.to(DEV), r.to(DEV), dz, dw, db, ws)
    d = f64(dy)
    h = (f64(z) - f64(m)[:, None]) * f64(r)[:, None]
    close(dw, (d * h).sum(0), (rows + 4) * U * np.abs(d * h).sum(0), "dweight")
    # a constant row is its own mean: no gradient of the weight at all
    z.fill_(mean)
    m.fill_(mean)
    sq.layer_norm_backward(dy.to(DEV), z.to(DEV), None, m.to(DEV), torch.full((rows,), 316.0, device=DEV), dz, dw,
                           db, ws)
    assert (dw == 0).all()
