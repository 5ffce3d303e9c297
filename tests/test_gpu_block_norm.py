"""Layer norm, its backward pass and dropout with the residual sum on the GPU, against their
64-bit definitions (oracle/block.py).

Tolerances, from the arithmetic: an output's last rounding is off by at most half a step,
eps / 2 of its type relative to the value (H below; fp16 adds half its smallest step).  Before it every
value is binary32 with U = 2^-24 per operation: a thread adds at most 8 * 16 values in sequence
(the longest rows: 8 * ceil(cols / 8192)), then 6 steps over a wave and 16 over its waves,
so a sum's error is at most S = 160 U times the sum of magnitudes for rows of up to 131072 elements.
"""
import numpy as np
import pytest
import torch

import oracle.block as OB
import scaled_quantization_amd as sq
from gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
S = 160 * U
TYPES = [torch.bfloat16, torch.float16, torch.float32]
IDS = ["bf16", "f16", "f32"]
# one vector, odd, and both sides of every change of threads or registers per row
COLS = [1, 7, 8, 9, 100, 511, 512, 513, 768, 1001, 1024, 1025, 2048, 2049, 4096, 4099, 8192, 8193,
        16384, 16385, 40001]
SEED, OFFSET = 0x123456789ABCDEF, 0x5_0000_0007


def half(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half the smallest step of type t (its subnormals' spacing)."""
    return {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}[t]


def draw(shape, t, seed, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(t)


def f64(x):
    return x.cpu().double().numpy()


def rng_words(seed=SEED, offset=OFFSET):
    return torch.tensor([seed, offset], dtype=torch.int64, device=DEV)


def close(got, ref, tol, what):
    got = f64(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {ref[bad][0]}, allowed {np.broadcast_to(tol, ref.shape)[bad][0]}")


def norm_tolerance(x, w, b, ref, mean, rstd, t):
    """Of y: the error of mean (S mean|x|) and of x - mean, relative to rstd; rstd's own (half the
    variance's: S, and the rounded distances), three products, one sum, the last rounding."""
    off = S * np.abs(x).mean(1) + U * np.abs(x).max(1)            # of x - mean
    rel = S + 2 * off * rstd + 8 * U                              # of rstd and the products
    h = np.abs(x - mean[:, None]) * rstd[:, None]
    e = np.abs(w) * (off[:, None] * rstd[:, None] + h * rel[:, None]) + U * np.abs(b)
    return e * (1 + half(t)) + half(t) * np.abs(ref) + tiny(t), off, rel


def check_norm(x, w, b, eps, y, mean, rstd, t, what):
    """y, mean, rstd of the kernel against the definition for float64 inputs."""
    ref, rmean, rrstd = OB.layer_norm(x, w, b, eps)
    tol, off, rel = norm_tolerance(x, w, b, ref, rmean, rrstd, t)
    close(y, ref, tol, what + " y")
    if mean is not None:
        close(mean, rmean, off + U * np.abs(rmean), what + " mean")
        close(rstd, rrstd, rel * rrstd, what + " rstd")


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_layer_norm(t, cols):
    rows = 5 if cols < 5000 else 3
    x = draw((rows, cols), t, cols, 1.5, 0.5)
    wt = t if cols % 2 else torch.float32
    w, b = draw(cols, wt, 1, 0.5, 1.0), draw(cols, wt, 2)
    y = torch.empty_like(x, device=DEV)
    mean, rstd = (torch.empty(rows, device=DEV) for _ in range(2))
    sq.layer_norm(x.to(DEV), w.to(DEV), b.to(DEV), 1e-5, y, mean, rstd)
    check_norm(f64(x), f64(w), f64(b), 1e-5, y, mean, rstd, t, f"{cols}")


@pytest.mark.parametrize("cols", [33, 768, 3000, 20000])
def test_layer_norm_without_parameters_and_many_rows(cols):
    # more rows than one pass of the grid takes; three dimensions; no mean, no rstd
    rows = 2 * 35003 if cols == 33 else 6
    x = draw((2, rows // 2, cols), torch.bfloat16, 3, 2.0)
    y = torch.empty_like(x, device=DEV)
    sq.layer_norm(x.to(DEV), None, None, 1e-6, y)
    check_norm(f64(x).reshape(rows, cols), np.ones(cols), np.zeros(cols), 1e-6,
               y.reshape(rows, cols), None, None, torch.bfloat16, "no parameters")


@pytest.mark.parametrize("cols", [100, 4096, 20000])
def test_layer_norm_row_that_is_not_finite_or_constant(cols):
    x = draw((5, cols), torch.bfloat16, 4)
    x[1, 3], x[2, 50], x[3] = float("nan"), float("inf"), 2.5
    y = torch.empty_like(x, device=DEV)
    sq.layer_norm(x.to(DEV), None, None, 1e-5, y)
    assert torch.isnan(y[1:3]).all() and (y[3] == 0).all()
    keep = [0, 4]
    check_norm(f64(x)[keep], np.ones(cols), np.zeros(cols), 1e-5, y[keep], None, None,
               torch.bfloat16, "the other rows")


def test_layer_norm_distant_mean():
    # mean 1000 standard deviations away: the variance does not cancel
    x = draw((4, 1536), torch.float32, 6, 1.0, 1000.0)
    y, mean, rstd = torch.empty_like(x, device=DEV), torch.empty(4, device=DEV), \
        torch.empty(4, device=DEV)
    sq.layer_norm(x.to(DEV), None, None, 1e-5, y, mean, rstd)
    check_norm(f64(x), np.ones(1536), np.zeros(1536), 1e-5, y, mean, rstd, torch.float32, "distant")


@pytest.mark.parametrize("off", [1, 3])
def test_tensors_that_start_at_any_element(off):
    # slices of a larger buffer: no 16-byte alignment anywhere
    rows, cols, t = 7, 1000, torch.bfloat16
    place = lambda v: torch.cat([torch.zeros(off, dtype=v.dtype), v.flatten()]).to(DEV)[off:].view(v.shape)
    x, w, b = draw((rows, cols), t, 7), draw(cols, t, 8, 0.2, 1.0), draw(cols, t, 9)
    y = place(torch.zeros_like(x))
    q, scale = place(torch.zeros((rows, cols), dtype=torch.int8)), torch.empty(rows, device=DEV)
    sq.layer_norm(place(x), place(w), place(b), 1e-5, y)
    check_norm(f64(x), f64(w), f64(b), 1e-5, y, None, None, t, "offset")
    sq.quantize_int8(place(x), q, scale)
    assert np.array_equal(q.cpu().numpy(), OB.quantize_int8(f64(x))[0])
    dz, dw, db = place(torch.zeros_like(x)), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    mean, rstd = x.float().mean(1).to(DEV), torch.ones(rows, device=DEV)
    ws = torch.empty(2 * rows * cols, device=DEV)
    sq.layer_norm_backward(place(x), place(x), place(w), mean, rstd, dz, dw, db, ws)
    check_backward(x, x, w, mean, rstd, None, dz, None, dw, db, t, "offset")


# ------------------------------------------------------------------ backward
def check_backward(dy, z, w, mean, rstd, add, dz, dx, dw, db, t, what, factor=None):
    d, x, w, m, r = f64(dy), f64(z), f64(w), f64(mean), f64(rstd)
    ref, rdw, rdb = OB.layer_norm_backward(d, x, w, m, r)
    h, g = np.abs((x - m[:, None]) * r[:, None]), np.abs(d * w)
    # h is off by 2 U + U (|x| + |m|) rstd, g by U, the two means by S of their terms' magnitudes
    eh = 2 * U * h + U * (np.abs(x) + np.abs(m[:, None])) * np.abs(r[:, None])
    mgh = (g * h).mean(1, keepdims=True)
    e = np.abs(r[:, None]) * (4 * U * g + S * g.mean(1, keepdims=True) + eh * mgh +
                              h * ((S + 4 * U) * mgh + (g * eh).mean(1, keepdims=True)) + 4 * U * h * mgh)
    if add is not None:
        ref = ref + f64(add)
        e = e + U * (np.abs(ref) + np.abs(f64(add)))
    close(dz, ref, e * (1 + half(t)) + half(t) * np.abs(ref) + tiny(t), what + " dz")
    if dx is not None:
        f = factor if factor is not None else np.ones_like(ref)
        close(dx, ref * f, (e + U * np.abs(ref)) * f * (1 + half(t)) + half(t) * np.abs(ref * f) + tiny(t),
              what + " dx")
    if dw is not None:
        # a column's sum: at most rows values in sequence in a thread, in a workgroup's tree and over
        # the parts; each order is covered by (rows + 40) U of the magnitudes
        n = (len(d) + 40) * U
        close(dw, rdw, n * (np.abs(d) * h).sum(0) + (np.abs(d) * eh).sum(0) + 1e-30, what + " dweight")
        close(db, rdb, n * np.abs(d).sum(0) + 1e-30, what + " dbias")


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_layer_norm_backward(t, cols):
    rows = 37 if cols < 5000 else 5
    z, dy = draw((rows, cols), t, cols, 1.5, 0.5), draw((rows, cols), t, cols + 1)
    w = draw(cols, torch.float32 if cols % 2 else t, 1, 0.5, 1.0)
    mean = z.float().mean(1)
    rstd = 1.0 / torch.sqrt(z.float().var(1, unbiased=False) + 1e-5)
    add = draw((rows, cols), t, cols + 2) if cols % 3 else None
    fused = cols % 4 != 0
    dz, dx = (torch.empty_like(z, device=DEV) for _ in range(2))
    dw, db = (torch.empty(cols, device=DEV) for _ in range(2))
    ws = torch.full((2 * rows * cols,), float("nan"), device=DEV)
    on = lambda v: None if v is None else v.to(DEV)
    sq.layer_norm_backward(on(dy), on(z), on(w), on(mean), on(rstd), dz, dw, db, ws, on(add), 0.3,
                           rng_words(), dx if fused else None)
    factor = OB.drop_factor(rows, cols, 0.3, SEED, OFFSET)
    check_backward(dy, z, w, mean, rstd, add, dz, dx if fused else None, dw, db, t, f"{cols}", factor)


@pytest.mark.parametrize("rows, cols", [(1, 768), (2, 768), (4097, 768), (9001, 64), (3001, 2048),
                                        (2500, 4096), (1100, 16384), (1500, 17000)])
def test_layer_norm_backward_rows(rows, cols):
    # more rows than the grid holds at once, in each form; the same call gives the same bits
    t = torch.bfloat16
    z, dy = draw((rows, cols), t, rows), draw((rows, cols), t, rows + 1)
    w = draw(cols, t, 1, 0.5, 1.0)
    mean, rstd = z.float().mean(1), 1.0 / torch.sqrt(z.float().var(1, unbiased=False) + 1e-5)
    args = [v.to(DEV) for v in (dy, z, w, mean, rstd)]
    ws = torch.empty(2 * min(rows, sq.NORM_PARTS) * cols, device=DEV)
    out = []
    for _ in range(2):
        dz = torch.empty_like(args[1])
        dw, db = (torch.empty(cols, device=DEV) for _ in range(2))
        sq.layer_norm_backward(*args, dz, dw, db, ws)
        out.append((dz, dw, db))
    assert all(torch.equal(a, b) for a, b in zip(*out))
    check_backward(dy, z, w, mean, rstd, None, *out[0][:1], None, *out[0][1:], t, f"{rows} rows")


def test_layer_norm_backward_in_place_and_without_sums():
    for cols in (768, 17000):      # dz over dy, dx over dz_add, in the form for short rows and for long
        t, rows = torch.bfloat16, 50
        z, dy, add = (draw((rows, cols), t, s) for s in (1, 2, 3))
        mean, rstd = z.float().mean(1), torch.ones(rows)
        d, a = dy.to(DEV), add.to(DEV)
        dw, db = (torch.empty(cols, device=DEV) for _ in range(2))
        ws = torch.empty(2 * rows * cols, device=DEV)
        sq.layer_norm_backward(d, z.to(DEV), None, mean.to(DEV), rstd.to(DEV), d, dw, db, ws, a, 0.5,
                               rng_words(), a)
        check_backward(dy, z, torch.ones(cols), mean, rstd, add, d, a, dw, db, t, "in place",
                       OB.drop_factor(rows, cols, 0.5, SEED, OFFSET))
        dz = torch.empty_like(d)
        sq.layer_norm_backward(dy.to(DEV), z.to(DEV), None, mean.to(DEV), rstd.to(DEV), dz)
        check_backward(dy, z, torch.ones(cols), mean, rstd, None, dz, None, None, None, t, "no sums")


def test_layer_norm_backward_against_differences():
    # the kernels' own forward in binary32: central differences of sum(y dy) along random directions.
    # y is off by at most 64 U of about 4, so the sums' difference by 2 * 64 U * 4 * sum|dy| at worst;
    # over a step of 2 * 2^-6 that and the third-order term (step^2 / 6 times a few) bound the gap
    rows, cols, step = 3, 40, 2.0 ** -6
    x, dy = draw((rows, cols), torch.float32, 1), draw((rows, cols), torch.float32, 2)
    w, b = draw(cols, torch.float32, 3, 0.3, 1.0), draw(cols, torch.float32, 4)

    def forward(x, w, b):
        y, m, r = torch.empty_like(x, device=DEV), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        sq.layer_norm(x.to(DEV), w.to(DEV), b.to(DEV), 1e-5, y, m, r)
        return y, m, r

    y, m, r = forward(x, w, b)
    dz, dw, db = torch.empty_like(y), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    sq.layer_norm_backward(dy.to(DEV), x.to(DEV), w.to(DEV), m, r, dz, dw, db,
                           torch.empty(2 * rows * cols, device=DEV))
    noise = 2 * 64 * U * 4 * float(dy.abs().sum()) / (2 * step)
    for seed in range(5, 8):
        dirs = [draw(v.shape, torch.float32, seed + 10 * i) for i, v in enumerate((x, w, b))]
        dirs = [d / d.norm() for d in dirs]
        for i, (d, grad) in enumerate(zip(dirs, (dz, dw, db))):
            ends = []
            for s in (step, -step):
                args = [x, w, b]
                args[i] = args[i] + s * d
                ends.append(float((f64(forward(*args)[0]) * f64(dy)).sum()))
            want = float((f64(grad) * f64(d)).sum())
            third = step ** 2 * 10 * float(dy.norm())
            assert abs((ends[0] - ends[1]) / (2 * step) - want) <= noise + third, (i, seed)


# ------------------------------------------------------------------ dropout
@pytest.mark.parametrize("cols", [1, 8, 13, 512, 1001, 2049, 8193, 20000])
@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_dropout_add(t, cols):
    rows = 9
    x, res = draw((rows, cols), t, 1), draw((rows, cols), t, 2)
    for p in (0.0, 0.1, 0.5, 1.0):
        f = OB.drop_factor(rows, cols, p, SEED, OFFSET)
        for r in (None, res):
            out = torch.empty_like(x, device=DEV)
            sq.dropout_add(x.to(DEV), None if r is None else r.to(DEV), p, rng_words() if p else None,
                           out)
            scaled = f64(x) * f
            ref = scaled + (0 if r is None else f64(r))
            close(out, ref, 2 * U * (np.abs(scaled) + np.abs(ref)) * (1 + half(t)) + half(t) * np.abs(ref) + tiny(t),
                  f"p {p}")
            if r is None:
                assert np.array_equal((f64(out) != 0), (f != 0) & (f64(x) != 0))


@pytest.mark.parametrize("rows, cols", [(1, 30_000_001), (30_000_001, 1), (70_001, 513), (3, 4_000_003)])
def test_dropout_add_long_or_many_rows(rows, cols):
    # more vectors than one pass of the grid takes, in one row, in rows of one element and between
    x = draw((rows, cols), torch.bfloat16, 1)
    out = torch.empty_like(x, device=DEV)
    sq.dropout_add(x.to(DEV), None, 0.5, rng_words(), out)
    f = OB.drop_factor(rows, cols, 0.5, SEED, OFFSET)
    assert np.array_equal(f64(out), f64(x) * f)


@pytest.mark.parametrize("cols", [300_001, 1_100_000])
def test_layer_norm_backward_very_long_rows(cols):
    t, rows = torch.bfloat16, 2
    z, dy = draw((rows, cols), t, 1), draw((rows, cols), t, 2)
    mean, rstd = z.float().mean(1), torch.ones(rows)
    dz, dw, db = torch.empty_like(z, device=DEV), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    sq.layer_norm_backward(dy.to(DEV), z.to(DEV), None, mean.to(DEV), rstd.to(DEV), dz, dw, db,
                           torch.empty(2 * rows * cols, device=DEV))
    d, h = f64(dy), f64(z) - f64(mean)[:, None]
    # dweight sees mean's rounding (U of z and mean) and three roundings per row
    close(dw, (d * h).sum(0), 8 * U * (np.abs(d) * (np.abs(h) + 1)).sum(0) + 1e-30, "dweight")
    close(db, d.sum(0), 2 * U * np.abs(d).sum(0) + 1e-30, "dbias")


def test_dropout_drops_what_is_not_finite_and_works_in_place():
    x = draw((4, 100), torch.bfloat16, 3)
    x[:, ::7] = float("inf")
    x[:, 1::7] = float("nan")
    f = OB.drop_factor(4, 100, 0.5, SEED, OFFSET)
    out = x.to(DEV)
    sq.dropout_add(out, None, 0.5, rng_words(), out)
    got, want = f64(out), OB.dropped(f64(x), f)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and (got[f == 0] == 0).all()
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])


@pytest.mark.parametrize("cols", [9, 768, 1001, 4096, 9000, 20001])
@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_dropout_add_layer_norm(t, cols):
    rows = 6
    x, res = draw((rows, cols), t, 1), draw((rows, cols), t, 2, 2.0)
    w, b = draw(cols, t, 3, 0.3, 1.0), draw(cols, t, 4)
    f = OB.drop_factor(rows, cols, 0.2, SEED, OFFSET)
    for p, r, factor in ((0.2, res, f), (0.0, res, np.ones_like(f)), (0.2, None, f)):
        z, y = (torch.empty_like(x, device=DEV) for _ in range(2))
        mean, rstd = (torch.empty(rows, device=DEV) for _ in range(2))
        sq.dropout_add_layer_norm(x.to(DEV), None if r is None else r.to(DEV), p,
                                  rng_words() if p else None, w.to(DEV), b.to(DEV), 1e-5, z, y, mean, rstd)
        scaled = f64(x) * factor
        ref = scaled + (0 if r is None else f64(r))
        close(z, ref, 2 * U * (np.abs(scaled) + np.abs(ref)) * (1 + half(t)) + half(t) * np.abs(ref) + tiny(t), "z")
        check_norm(f64(z), f64(w), f64(b), 1e-5, y, mean, rstd, t, "norm of z as stored")
    # z may be the residual's buffer, and the mask is dropout_add's
    z2, y2 = res.to(DEV), torch.empty_like(x, device=DEV)
    sq.dropout_add_layer_norm(x.to(DEV), z2, 0.2, rng_words(), w.to(DEV), b.to(DEV), 1e-5, z2, y2)
    alone = torch.empty_like(z2)
    sq.dropout_add(x.to(DEV), res.to(DEV), 0.2, rng_words(), alone)
    assert torch.equal(z2, alone)


def test_offsets_past_32_bits():
    # 70001 x 32768 elements (2.3 G): sampled rows at the end against the definition
    rows, cols, t = 70001, 32768, torch.bfloat16
    x = torch.empty((rows, cols), dtype=t, device=DEV)
    index = [0, 65535, 65536, 69999, 70000]
    some = draw((len(index), cols), t, 1)
    x.fill_(1.0)
    x[index] = some.to(DEV)
    out = torch.empty_like(x)
    sq.dropout_add(x, None, 0.5, rng_words(), out)
    f = OB.drop_factor(index, cols, 0.5, SEED, OFFSET)
    assert np.array_equal(f64(out[index]), f64(some) * f)
    mean, rstd = (torch.empty(rows, device=DEV) for _ in range(2))
    sq.layer_norm(x, None, None, 1e-5, out, mean, rstd)
    check_norm(f64(some), np.ones(cols), np.zeros(cols), 1e-5, out[index], mean[index], rstd[index], t, "far")
    dz, dw, db = torch.empty_like(x), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    sq.layer_norm_backward(out, x, None, mean, rstd, dz, dw, db,
                           torch.empty(2 * sq.NORM_PARTS * cols, device=DEV))
    check_backward(out[index], some, torch.ones(cols), mean[index], rstd[index], None, dz[index], None, None,
                   None, t, "far")
    # rows of ones have h = 0 and dy = 0: only the sampled rows reach the sums
    d, h = f64(out[index]), (f64(some) - f64(mean[index])[:, None]) * f64(rstd[index])[:, None]
    close(dw, (d * h).sum(0), 64 * U * (np.abs(d * h)).sum(0) + 1e-6, "far dweight")
    close(db, d.sum(0), 64 * U * np.abs(d).sum(0) + 1e-6, "far dbias")


# ------------------------------------------------------------------ streams and graphs
def test_side_stream_and_graph_replays():
    rows, cols, t = 300, 768, torch.bfloat16
    x, res, dy = (draw((rows, cols), t, s).to(DEV) for s in (1, 2, 3))
    w, b = draw(cols, t, 4, 0.3, 1.0).to(DEV), draw(cols, t, 5).to(DEV)
    rng = rng_words()

    def buffers():
        big = lambda: torch.empty_like(x)
        return dict(z=big(), y=big(), mean=torch.empty(rows, device=DEV), rstd=torch.empty(rows, device=DEV),
                    dz=big(), dx=big(), dw=torch.empty(cols, device=DEV), db=torch.empty(cols, device=DEV),
                    ws=torch.empty(2 * rows * cols, device=DEV))

    def step(o):
        sq.dropout_add_layer_norm(x, res, 0.3, rng, w, b, 1e-5, o["z"], o["y"], o["mean"], o["rstd"])
        sq.layer_norm_backward(dy, o["z"], w, o["mean"], o["rstd"], o["dz"], o["dw"], o["db"], o["ws"],
                               None, 0.3, rng, o["dx"])

    eager, side, graphed = buffers(), buffers(), buffers()
    step(eager)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step(graphed)
    torch.cuda.synchronize()
    names = [n for n in eager if n != "ws"]
    assert all(torch.equal(eager[n], side[n]) for n in names)
    for i in range(4):              # the offset moves between replays: another mask each time
        rng[1] += 1
        x.add_(0.125)
        g.replay()
        torch.cuda.synchronize()
        before = eager["z"].clone()
        step(eager)
        torch.cuda.synchronize()
        assert all(torch.equal(eager[n], graphed[n]) for n in names), i
        assert not torch.equal(before, eager["z"])


def test_refusals_on_the_device():
    x = torch.zeros((4, 16), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(sq.Fp8dpError, match="contiguous"):
        sq.layer_norm(x[:, :8], None, None, 1e-5, torch.empty((4, 8), dtype=x.dtype, device=DEV))
    with pytest.raises(sq.Fp8dpError, match="rows"):
        sq.layer_norm(x[:0], None, None, 1e-5, x[:0])
    with pytest.raises(sq.Fp8dpError, match="rng"):
        sq.dropout_add(x, None, 0.5, None, x)
    with pytest.raises(sq.Fp8dpError, match="same buffer"):
        sq.dropout_add_layer_norm(x, None, 0.0, None, None, None, 1e-5, x, x)
