"""Where the operators around the MLP keep more than their outputs' own rounding (GPU): INT8 codes
behind a norm, weight gradients of rows far from zero, sums over very long rows and very many.

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


# ------------------------------------------------------------------ long sums
# Off by at most L U of the terms' magnitudes, whatever their number: 3 additions of a vector's 8 values, 2 of
# the compensated sum of a thread's vectors, 6 over a wave, 16 over its waves, the division's 2, the terms' own 3.
L = 32 * U


def near(shape, seed, std):
    """Nearly equal float32 values: a plain running sum rounds them all to the same side for long."""
    return 1.1 + std * draw(shape, torch.float32, seed)


@pytest.mark.parametrize("cols", [100_003, 4_000_001, 1 << 25])
def test_norm_of_very_long_rows(cols):
    x = near((2, cols), 1, 1e-3)
    y = torch.empty_like(x, device=DEV)
    mean, rstd = torch.empty(2, device=DEV), torch.empty(2, device=DEV)
    sq.layer_norm(x.to(DEV), None, None, 0.0, y, mean, rstd)
    ref, m, r = OB.layer_norm(f64(x), 1.0, 0.0, 0.0)
    off = L * np.abs(f64(x)).mean(1)                 # of the mean, and of x - mean
    close(mean, m, off, "mean")
    # the variance is off by 2 off mean|x - mean| <= 2 off / rstd and L of itself, and rstd by half of that
    rel = off * r + L
    close(rstd, r, rel * r, "rstd")
    close(y, ref, ((off * r)[:, None] + np.abs(ref) * (rel[:, None] + 4 * U)), "y")


@pytest.mark.parametrize("cols", [100_003, 4_000_001, 1 << 24])
def test_gradient_of_very_long_rows(cols):
    # g = dy nearly constant: what is left of g - mean(g) shows the sum's error
    z, dy = draw((2, cols), torch.float32, 1), near((2, cols), 2, 1e-5)
    m, r = torch.zeros(2), torch.ones(2)
    dz = torch.empty_like(z, device=DEV)
    sq.layer_norm_backward(dy.to(DEV), z.to(DEV), None, m.to(DEV), r.to(DEV), dz)
    d, h = f64(dy), f64(z)
    mg, mgh = d.mean(1, keepdims=True), (d * h).mean(1, keepdims=True)
    tol = L * (np.abs(d).mean(1, keepdims=True) + np.abs(h) * np.abs(d * h).mean(1, keepdims=True)) + \
        4 * U * (np.abs(d) + np.abs(mg) + np.abs(h * mgh))
    close(dz, d - mg - h * mgh, tol, "dz")


# Down the rows a thread sums 64 of them plainly, and those sums again; the last bound is of (rows, cols) =
# (2^24, 8): 4096 rows a wave are 64 such sums.  Rows of less than a vector (or more than 8192 columns) go by a
# compensated sum.  3 more of each term, 2 over a workgroup's waves, 16 + 8 + 8 of the parts (64 ranges of at most
# 16, then two of 8).
@pytest.mark.parametrize("rows, cols, n", [(1 << 23, 4, 2), (1 << 24, 1, 2), ((1 << 22) + 3, 7, 2),
                                           (1 << 24, 8, 64 + 64), ((1 << 21) + 5, 100, 64 + 64)])
def test_weight_gradient_of_very_many_rows(rows, cols, n):
    z, dy = near((rows, cols), 1, 1e-5), near((rows, cols), 2, 1e-5)
    m, r = torch.zeros(rows, device=DEV), torch.ones(rows, device=DEV)
    dz, dw, db = torch.empty_like(z, device=DEV), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    ws = torch.empty(2 * sq.NORM_PARTS * cols, device=DEV)
    sq.layer_norm_backward(dy.to(DEV), z.to(DEV), None, m, r, dz, dw, db, ws)
    d, h = f64(dy), f64(z)
    close(dw, (d * h).sum(0), (n + 37) * U * np.abs(d * h).sum(0), "dweight")
    close(db, d.sum(0), (n + 37) * U * np.abs(d).sum(0), "dbias")


@pytest.mark.parametrize("cols", [4, 20, 20000])
def test_sums_that_are_not_finite(cols):
    # an infinite gradient leaves its column's sums infinite, a NaN makes them NaN; nothing else changes
    rows = 300
    z, dy = draw((rows, cols), torch.float32, 1), draw((rows, cols), torch.float32, 2)
    dy[7, 0], dy[200, 1], dy[9, 2] = float("inf"), -float("inf"), float("nan")
    m, r = torch.zeros(rows, device=DEV), torch.ones(rows, device=DEV)
    dz, dw, db = torch.empty_like(z, device=DEV), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    sq.layer_norm_backward(dy.to(DEV), z.to(DEV), None, m, r, dz, dw, db,
                           torch.empty(2 * rows * cols, device=DEV))
    want = [float("inf"), -float("inf")]
    assert db[:2].tolist() == want and db[2].isnan() and db[3:].isfinite().all()
    assert dw[:2].tolist() == [w * float(z[i, c].sign()) for w, i, c in zip(want, (7, 200), (0, 1))]
    assert dw[2].isnan() and dw[3:].isfinite().all()
    bad = ~dz.isfinite()           # (mean(g) and mean(g h) are not, and reach every element of their rows)
    assert bad[[7, 9, 200]].all() and bad.sum() == 3 * cols
    # a row that holds an infinity is NaN whatever its length
    x = dy[:3].clone()
    x[1, 3] = float("inf")
    y = torch.empty_like(x, device=DEV)
    sq.layer_norm(x.to(DEV), None, None, 1e-5, y)
    assert y[1].isnan().all() and y[[0, 2]].isfinite().all()
