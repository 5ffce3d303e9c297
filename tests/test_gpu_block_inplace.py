"""The in-place forms of the operators around the MLP, at widths whose last vector is cut, and rows that are
not finite in the backward pass (GPU): bit for bit what separate buffers and finite neighbours give."""
import pytest
import torch

import scaled_quantization_amd as sq
from gpu_util import DEV
from test_gpu_block_norm import IDS, TYPES, draw, rng_words

pytestmark = pytest.mark.gpu

COLS = [7, 9, 100, 520, 768, 1001, 2049, 4099, 8195, 16390, 20001]


def many(cols):
    """Rows: several for every wave or workgroup of the grid where they are short."""
    return 9001 if cols <= 1024 else 1500 if cols < 5000 else 40


def same(a, b, what):
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), what


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_forward_in_place(t, cols):
    rows = many(cols)
    x, res = draw((rows, cols), t, 1).to(DEV), draw((rows, cols), t, 2).to(DEV)
    w, b, rng = draw(cols, t, 3, 0.3, 1.0).to(DEV), draw(cols, t, 4).to(DEV), rng_words()

    def run(x, res, z):
        y, mean, rstd = torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        sq.dropout_add_layer_norm(x, res, 0.3, rng, w, b, 1e-5, z, y, mean, rstd)
        return z, y, mean, rstd

    for r in (res, None):
        want = run(x, r, torch.empty_like(x))
        own = x.clone()
        for got, ref in zip(run(own, r, own), want):
            same(got, ref, "z over x")
        if r is not None:
            own = res.clone()
            for got, ref in zip(run(x, own, own), want):
                same(got, ref, "z over the residual")
        alone = torch.empty_like(x)
        sq.dropout_add(x, r, 0.3, rng, alone)
        same(alone, want[0], "dropout_add")
        for over_x in (True, False)[:1 if r is None else 2]:
            own = (x if over_x else r).clone()
            sq.dropout_add(own if over_x else x, r if over_x else own, 0.3, rng, own)
            same(own, alone, "out over x" if over_x else "out over the residual")


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_backward_in_place(t, cols):
    rows = many(cols)
    z, dy, add = (draw((rows, cols), t, s).to(DEV) for s in (1, 2, 3))
    w, rng = draw(cols, t, 4, 0.3, 1.0).to(DEV), rng_words()
    mean, rstd = z.float().mean(1), torch.rsqrt(z.float().var(1, unbiased=False) + 1e-5)
    ws = torch.empty(2 * min(rows, sq.NORM_PARTS) * cols, device=DEV)

    def run(dz, dx):
        """dz, dx: "dy", "add" or None for a buffer of its own."""
        have = {"dy": dy.clone(), "add": add.clone()}
        oz, ox = (have[k] if k else torch.empty_like(z) for k in (dz, dx))
        dw, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
        sq.layer_norm_backward(have["dy"], z, w, mean, rstd, oz, dw, db, ws, have["add"], 0.3, rng, ox)
        return oz, ox, dw, db

    want = run(None, None)
    for names in (("dy", None), ("add", None), (None, "dy"), (None, "add"), ("dy", "add"), ("add", "dy")):
        for got, ref in zip(run(*names), want):
            same(got, ref, f"dz over {names[0]}, dx over {names[1]}")


@pytest.mark.parametrize("cols", [7, 100, 768, 1001, 4099, 8195, 20001])
@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_rows_that_are_not_finite_leave_the_others(t, cols):
    rows = 4500 if cols <= 1024 else 60
    z, dy, add = (draw((rows, cols), t, s).to(DEV) for s in (1, 2, 3))
    nan, inf = float("nan"), float("inf")
    bad = [0, 5, 33, rows - 1]

    def run(z, dy):
        mean, rstd = z.float().mean(1), torch.rsqrt(z.float().var(1, unbiased=False) + 1e-5)
        dz, dx = torch.empty_like(z), torch.empty_like(z)
        dw, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
        sq.layer_norm_backward(dy, z, None, mean, rstd, dz, dw, db,
                               torch.empty(2 * min(rows, sq.NORM_PARTS) * cols, device=DEV), add, 0.5,
                               rng_words(), dx)
        return dz, dx, dw, db

    fine = run(z, dy)
    z2, dy2 = z.clone(), dy.clone()
    z2[bad[0], cols - 1], z2[bad[1], 0] = nan, -inf
    dy2[bad[2], cols - 1], dy2[bad[3], 2] = nan, inf
    dz, dx, dw, db = run(z2, dy2)
    keep = torch.ones(rows, dtype=torch.bool, device=DEV)
    keep[bad] = False
    same(dz[keep], fine[0][keep], "dz of the other rows")
    same(dx[keep], fine[1][keep], "dx of the other rows")
    assert not dz[~keep].isfinite().any()
    assert (dx[~keep] == 0).any() and not dx[~keep][dx[~keep] != 0].isfinite().any()    # dropped: +0
    # z's two rows have no finite h, so no column of dweight is; dbias sees dy alone
    assert not dw.isfinite().any()
    assert db[cols - 1].isnan() and db[2] == inf and db.isfinite().sum() == cols - 2
