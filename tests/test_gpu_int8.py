"""INT8 codes per row, the INT8 product and the linear layer on the GPU, against their 64-bit
definitions (oracle/block.py).

Codes of tensors are equal to the definition's.  A product's sums are exact; what is rounded is the sum's
conversion, two products and one sum in binary32 (U = 2^-24 each), then the output's type
(eps / 2 of the value, half its smallest step at least)."""
import numpy as np
import pytest
import torch

import oracle.block as OB
import scaled_quantization_amd as sq
from gpu_util import DEV
from test_gpu_block_norm import IDS, TYPES, U, close, draw, f64, half, norm_tolerance, tiny

pytestmark = pytest.mark.gpu


def codes_of(x, what=""):
    q = torch.empty(x.shape, dtype=torch.int8, device=DEV)
    scale = torch.empty(x.numel() // x.shape[-1], device=DEV)
    sq.quantize_int8(x.to(DEV), q, scale)
    return q, scale


@pytest.mark.parametrize("cols", [1, 7, 8, 9, 100, 512, 513, 1000, 1024, 1025, 2048, 2050, 4096, 4100,
                                  8192, 8200, 16384, 16390, 33333])
@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_quantize_int8(t, cols):
    rows = 11 if cols < 5000 else 4
    x = draw((rows, cols), t, cols)
    x[0] = x[0].abs().max() * torch.randint(-254, 255, (cols,)) / 254     # ties in plenty
    q, scale = codes_of(x)
    want, s = OB.quantize_int8(f64(x))
    assert np.array_equal(q.cpu().numpy(), want)
    close(scale, s, U * s, "scale")


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_quantize_int8_every_16_bit_value(t):
    # every finite value under many maxima: 2^16 patterns per row (binary32: patterns of bf16 with noise)
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    if t == torch.float32:
        vals = bits.view(torch.bfloat16).float()
        vals = vals * (1 + 1e-4 * draw(65536, t, 1))
    else:
        vals = bits.view(t).clone()
    vals = torch.where(torch.isfinite(vals), vals, torch.zeros_like(vals))
    fin = torch.finfo(t)
    tops = torch.tensor([fin.max, fin.tiny, fin.smallest_normal * 3, 1.0, 1.5, 3.0, 127.0, 254.0, 0.7,
                         1e-3, 333.0, 2.0 ** -13])
    rows = []
    for top in tops.to(t):
        rows.append(vals.clamp(-top.item(), top.item()))
        rows[-1][0] = top
    x = torch.stack(rows)
    q, scale = codes_of(x)
    want, _ = OB.quantize_int8(f64(x))
    assert np.array_equal(q.cpu().numpy(), want)


@pytest.mark.parametrize("cols", [5, 700, 4096, 20000])
def test_quantize_int8_rows_of_zeros_and_rows_that_are_not_finite(cols):
    x = draw((6, cols), torch.bfloat16, 1)
    x[1] = 0
    x[2, 0], x[3, cols - 1], x[4, cols // 2] = float("inf"), float("nan"), -float("inf")
    q, scale = codes_of(x)
    assert (q[1:5] == 0).all() and scale[1] == 0 and torch.isnan(scale[2:5]).all()
    keep = [0, 5]
    assert np.array_equal(q[keep].cpu().numpy(), OB.quantize_int8(f64(x)[keep])[0])
    # a product with such a row: zeros stay the bias, the others are NaN, the rest is untouched
    w8 = torch.randint(-127, 128, (40, cols), dtype=torch.int8, device=DEV)
    y = torch.empty((6, 40), device=DEV)
    sq.int8_gemm(q, w8, scale, torch.ones(40, device=DEV), y, torch.full((40,), 3.0, device=DEV))
    assert (y[1] == 3).all() and torch.isnan(y[2:5]).all() and torch.isfinite(y[keep]).all()


@pytest.mark.parametrize("cols", [8, 100, 768, 1001, 4096, 8200, 20000])
@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_layer_norm_quantize_int8(t, cols):
    rows = 7
    x, res = draw((rows, cols), t, 1, 2.0, 0.5), draw((rows, cols), t, 2)
    w, b = draw(cols, t, 3, 0.3, 1.0), draw(cols, t, 4, 0.2)
    q = torch.empty((rows, cols), dtype=torch.int8, device=DEV)
    scale = torch.empty(rows, device=DEV)
    for r in (None, res):
        z = None if r is None else torch.empty_like(x, device=DEV)
        sq.layer_norm_quantize_int8(x.to(DEV), w.to(DEV), b.to(DEV), 1e-5, q, scale,
                                    None if r is None else r.to(DEV), z)
        v = f64(x)
        if r is not None:
            both = f64(x) + f64(r)
            close(z, both, U * np.abs(both) + half(t) * np.abs(both) + tiny(t), "z")
            v = f64(z)
        ref, mean, rstd = OB.layer_norm(v, f64(w), f64(b), 1e-5)
        # the norm's own error before the cast, as of a binary32 output; half a code; the scale's error
        e, _, _ = norm_tolerance(v, f64(w), f64(b), ref, mean, rstd, torch.float32)
        top = np.abs(ref).max(1)
        close(scale, top / 127, (e.max(1) + 2 * U * top) / 127, "scale")
        s = f64(scale)[:, None]
        close(torch.from_numpy(f64(q) * s), ref, s / 2 + e + 2 * e.max(1)[:, None] + 4 * U * np.abs(ref), "codes")
        assert (np.abs(f64(q)).max(1) == 127).all()


# ------------------------------------------------------------------ product
def operands(M, N, K, seed, full=False):
    rng = np.random.default_rng(seed)
    a = rng.integers(-128, 128, (M, K), dtype=np.int8)
    b = rng.integers(-128, 128, (N, K), dtype=np.int8)
    if full:
        a[:] = -128
        b[:] = -128
    return a, b, rng.uniform(0.001, 0.02, M).astype(np.float32), rng.uniform(0.001, 0.02, N).astype(np.float32)


def check_product(y, a, b, sa, sb, bias, t, what, rows=None):
    if rows is not None:
        a, sa, y = a[rows], sa[rows], y[rows]
    ref, sums = OB.int8_gemm(a, b, sa.astype(np.float64), sb.astype(np.float64), bias)
    mag = np.abs(sums * sa[:, None].astype(np.float64) * sb) + (0 if bias is None else np.abs(bias))
    close(y, ref, 5 * U * mag + half(t) * np.abs(ref) + tiny(t), what)


SHAPES = [(1, 1, 1), (1, 4096, 4096), (2, 17, 15), (3, 64, 16), (5, 130, 129), (16, 256, 128), (17, 250, 1000), (5, 60, 1040), (40, 100, 400),
          (33, 50, 272), (12, 33, 2064), (60, 17, 4240),
          (31, 1023, 777), (48, 512, 4096), (64, 64, 64), (65, 129, 257), (100, 300, 2000), (128, 128, 128),
          (129, 4, 4096), (200, 1000, 4112), (256, 256, 256), (257, 255, 1024), (300, 2049, 640),
          (512, 768, 1536), (777, 1023, 1001), (1000, 40, 32), (1024, 2304, 768), (2048, 512, 144),
          (2500, 1281, 528)]


@pytest.mark.parametrize("M, N, K", SHAPES)
def test_int8_gemm(M, N, K):
    a, b, sa, sb = operands(M, N, K, M + N + K)
    dev = [torch.from_numpy(v).to(DEV) for v in (a, b, sa, sb)]
    ws = torch.empty(16 << 20, dtype=torch.uint8, device=DEV)
    got = {}
    for i, t in enumerate(TYPES):
        for bt in (None, t, torch.float32):
            bias = None if bt is None else draw(N, bt, 3)
            for w in (None, ws):
                y = torch.full((M, N), float("nan"), dtype=t, device=DEV)
                sq.int8_gemm(*dev, y, None if bias is None else bias.to(DEV), w)
                check_product(y, a, b, sa, sb, None if bias is None else f64(bias), t,
                              f"{IDS[i]}, bias {bt}, workspace {w is not None}")
                key = (t, bt)
                assert key not in got or torch.equal(got[key], y)      # exact sums: the split changes nothing
                got[key] = y


@pytest.mark.parametrize("M, N, K", [(5, 40, 2000), (70, 70, 131071), (300, 300, 4096)])
def test_int8_gemm_largest_sums(M, N, K):
    a, b, sa, sb = operands(M, N, K, 1, full=True)
    dev = [torch.from_numpy(v).to(DEV) for v in (a, b, sa, sb)]
    y = torch.empty((M, N), device=DEV)
    sq.int8_gemm(*dev, y, None, torch.empty(16 << 20, dtype=torch.uint8, device=DEV))
    check_product(y, a, b, sa, sb, None, torch.float32, "all -128")


def test_int8_product_with_copied_operands():
    # rows at any byte and enough work: with a workspace both operands are copied to aligned rows
    # (int8_linear: the weight alone), without one they are not; the sums are the same
    M, N, K = 4200, 2100, 1901
    a, b, sa, sb = operands(M, N, K, 9)
    dev = [torch.from_numpy(v).to(DEV) for v in (a, b, sa, sb)]
    ys = []
    for room in (0, (M + N) * 1904, (M + N) * 1904 - 1, 1 << 25):
        y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
        sq.int8_gemm(*dev, y, None, torch.full((room,), 0x33, dtype=torch.uint8, device=DEV) if room else None)
        ys.append(y)
    assert all(torch.equal(ys[0], y) for y in ys[1:])
    rows = np.array([0, 1, 63, 64, 255, 256, 2047, 4095, 4096, 4198, 4199])
    check_product(ys[0], a, b, sa, sb, None, torch.bfloat16, "copied", rows)
    x = draw((M, K), torch.bfloat16, 1)
    need = sq.int8_linear_workspace(M, K)
    out = []
    for room in (need, need + N * 1904):
        y = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
        sq.int8_linear(x.to(DEV), dev[1], dev[3], y, torch.full((room,), 0x33, dtype=torch.uint8, device=DEV))
        out.append(y)
    assert torch.equal(*out)
    q, s = OB.quantize_int8(f64(x)[rows])
    check_product(out[0][torch.from_numpy(rows).to(DEV)], q, b, s.astype(np.float32), sb, None, torch.bfloat16,
                  "linear, copied")


@pytest.mark.parametrize("off", [1, 4, 8])
def test_int8_gemm_operands_that_start_at_any_byte(off):
    for M, N, K in ((33, 70, 256), (300, 260, 512), (3, 64, 1024)):
        a, b, sa, sb = operands(M, N, K, off)
        place = lambda v: torch.cat([torch.zeros(off, dtype=torch.int8), torch.from_numpy(v).flatten()]) \
            .to(DEV)[off:].view(v.shape)
        y = torch.empty(M * N + 1, dtype=torch.bfloat16, device=DEV)[1:].view(M, N)
        sq.int8_gemm(place(a), place(b), torch.from_numpy(sa).to(DEV), torch.from_numpy(sb).to(DEV), y)
        check_product(y, a, b, sa, sb, None, torch.bfloat16, f"offset {off}")


def test_int8_gemm_writes_nothing_beyond_y():
    for M, N, K in ((5, 33, 100), (65, 127, 256), (300, 259, 512), (1, 1000, 64)):
        a, b, sa, sb = operands(M, N, K, 2)
        y = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
        sq.int8_gemm(*(torch.from_numpy(v).to(DEV) for v in (a, b, sa, sb)), y[32:32 + M * N].view(M, N))
        assert (y[:32] == 7).all() and (y[32 + M * N:] == 7).all()
        check_product(y[32:32 + M * N].view(M, N), a, b, sa, sb, None, torch.bfloat16, f"{M} {N} {K}")


def test_int8_gemm_rows_past_32_bits():
    # a of 2.7 GB and y past 2^31 bytes: sampled rows
    M, N, K = 660_000, 2048, 4096
    rng = np.random.default_rng(3)
    index = np.array([0, 1, 255, 524287, 524288, 525001, 659_999])
    a = torch.ones((M, K), dtype=torch.int8, device=DEV)
    some, b, _, sb = operands(len(index), N, K, 4)
    a[torch.from_numpy(index).to(DEV)] = torch.from_numpy(some).to(DEV)
    sa = torch.full((M,), 0.01, device=DEV)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    sq.int8_gemm(a, torch.from_numpy(b).to(DEV), sa, torch.from_numpy(sb).to(DEV), y)
    check_product(y[torch.from_numpy(index).to(DEV)], some, b, np.full(len(index), 0.01, np.float32), sb, None,
                  torch.bfloat16, "far rows")


# ------------------------------------------------------------------ linear layer
@pytest.mark.parametrize("M, N, K", [(1, 4096, 4096), (1, 17, 5), (2, 300, 4096), (3, 1000, 2048),
                                     (4, 512, 4096), (4, 64, 16), (2, 33, 144), (1, 40, 16384), (1, 20, 65536),
                                     (3, 17, 1040), (4, 1000, 3000), (5, 50, 1024), (8, 300, 2048),
                                     (9, 40, 400), (16, 128, 1024), (13, 70, 272), (8, 256, 8192), (16, 512, 1001),
                                     (17, 512, 512), (48, 4096, 4096), (129, 1000, 1000), (777, 1023, 1001),
                                     (1500, 1024, 2048)])
@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_int8_linear(t, M, N, K):
    x, w = draw((M, K), t, 1), draw((N, K), t, 2, 0.02)
    bias = draw(N, t, 3)
    w8, w_scale = codes_of(w)
    need = sq.int8_linear_workspace(M, K)
    ys = []
    for room in (need, need + (16 << 20)):
        ws = torch.full((room,), 0x55, dtype=torch.uint8, device=DEV)
        y = torch.full((M, N), float("nan"), dtype=t, device=DEV)
        sq.int8_linear(x.to(DEV), w8, w_scale, y, ws, bias.to(DEV))
        ys.append(y)
    assert torch.equal(*ys)
    q, s = OB.quantize_int8(f64(x))
    s32 = s.astype(np.float32)
    check_product(ys[0], q, w8.cpu().numpy(), s32, f64(w_scale).astype(np.float32), f64(bias), t, "linear")
    # the same as its two parts
    q, scale = codes_of(x)
    y = torch.empty_like(ys[0])
    sq.int8_gemm(q, w8, scale, w_scale, y, bias.to(DEV))
    assert torch.equal(y, ys[0])


def test_int8_linear_row_that_is_not_finite():
    for M in (1, 2, 3, 4, 7, 16, 40):
        x = draw((M, 512), torch.bfloat16, 1)
        x[M - 1, 7] = float("nan")
        w8, w_scale = codes_of(draw((64, 512), torch.bfloat16, 2))
        y = torch.empty((M, 64), dtype=torch.bfloat16, device=DEV)
        sq.int8_linear(x.to(DEV), w8, w_scale, y,
                       torch.empty(sq.int8_linear_workspace(M, 512), dtype=torch.uint8, device=DEV))
        assert torch.isnan(y[M - 1]).all() and torch.isfinite(y[:M - 1]).all()


def test_int8_linear_graph_replays_and_side_stream():
    shapes = [(1, 512, 1024), (40, 300, 2048), (300, 512, 768)]
    state = []
    for M, N, K in shapes:
        w8, w_scale = codes_of(draw((N, K), torch.bfloat16, 2))
        new = lambda: (torch.empty((M, N), dtype=torch.bfloat16, device=DEV),
                       torch.empty(sq.int8_linear_workspace(M, K) + (16 << 20), dtype=torch.uint8, device=DEV))
        state.append((draw((M, K), torch.bfloat16, 1).to(DEV), w8, w_scale, new(), new()))

    def run(i):
        for x, w8, w_scale, *out in state:
            sq.int8_linear(x, w8, w_scale, *out[i])

    run(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(1)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            run(1)
    torch.cuda.synchronize()
    for i in range(4):
        for x, *_ in state:
            x.mul_(-0.5)
        g.replay()
        torch.cuda.synchronize()
        run(0)
        torch.cuda.synchronize()
        assert all(torch.equal(out[0][0], out[1][0]) for *_, a, b in state for out in ((a, b),)), i


def test_refusals_on_the_device():
    a = torch.zeros((4, 32), dtype=torch.int8, device=DEV)
    one = torch.ones(4, device=DEV)
    with pytest.raises(sq.Fp8dpError, match="contiguous"):
        sq.int8_gemm(a[:, :16], a[:, :16].contiguous(), one, one, torch.empty((4, 4), device=DEV))
    with pytest.raises(sq.Fp8dpError, match="must be"):
        sq.int8_gemm(a[:0], a, one[:0], one, torch.empty((0, 4), device=DEV))
    x = torch.zeros((4, 32), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(sq.Fp8dpError, match="workspace needs"):
        sq.int8_linear(x, a, one, torch.empty((4, 4), dtype=x.dtype, device=DEV),
                       torch.empty(100, dtype=torch.uint8, device=DEV))
