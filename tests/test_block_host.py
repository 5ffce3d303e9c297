"""The operators around the MLP without a GPU: the oracle against published and independent
values, the C ABI's symbols and refusals, and the binding's checks of its tensors.  No call
here reaches a GPU."""
import os
import re
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle.block as OB
import scaled_quantization_amd as sq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8dp_block.h")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(sq.LIB_PATH):
        pytest.skip("libfp8dp.so not built")
    return sq.lib()


# ------------------------------------------------------------------ oracle
@pytest.mark.parametrize("counter, key, want", [
    # known answers published with the generator (4 x 32 bits, 10 rounds)
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, want):
    assert tuple(int(w) for w in OB.philox4x32(counter, key)) == want


def test_drop_factor_mean_and_independence():
    # 4 Mi numbers: the kept share is binomial, 6 standard deviations off at most;
    # another offset or seed gives another mask
    f = OB.drop_factor(1024, 4096, 0.25, 3, 9)
    n, keep = f.size, (f != 0).mean()
    assert abs(keep - 0.75) < 6 * (0.75 * 0.25 / n) ** 0.5
    assert f.max() == 65536 / 49152
    for seed, offset in ((4, 9), (3, 10), (3, 9 + (1 << 32)), (3 + (1 << 32), 9)):
        g = OB.drop_factor(64, 4096, 0.25, seed, offset)
        same = ((g != 0) == (f[:64] != 0)).mean()
        assert abs(same - (0.75 ** 2 + 0.25 ** 2)) < 0.01


def test_quantize_oracle_is_exact():
    # against rational arithmetic, ties among them (x = amax / 2 gives 63.5, 3 / 254 amax 1.5)
    rng = np.random.default_rng(5)
    for top in (1.0, 3.0, 254.0, 1e-30, 3.1e38):
        t = np.float32(top)
        x = np.concatenate([[t, t / 2, -t / 2, t / 4], (rng.uniform(-1, 1, 60) * t),
                            t * np.arange(1, 40, 2) / 254]).astype(np.float32)
        q, s = OB.quantize_int8(x[None, :].astype(np.float64))
        for v, c in zip(x.tolist(), q[0].tolist()):
            assert round(Fraction(v) * 127 / Fraction(float(t))) == c     # Python rounds ties to even
        assert s[0] == float(t) / 127


def test_layer_norm_gradient_oracle_against_differences():
    rng = np.random.default_rng(8)
    x, w, b = rng.normal(size=(3, 11)) * 2 + 1, rng.normal(size=11), rng.normal(size=11)
    dy = rng.normal(size=(3, 11))
    eps, step = 1e-5, 1e-6
    _, mean, rstd = OB.layer_norm(x, w, b, eps)
    dz, dw, db = OB.layer_norm_backward(dy, x, w, mean, rstd)

    def loss(x, w, b):
        return (OB.layer_norm(x, w, b, eps)[0] * dy).sum()

    def differences(v, f):
        out = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            up, down = v.copy(), v.copy()
            up[i] += step
            down[i] -= step
            out[i] = (f(up) - f(down)) / (2 * step)
        return out

    np.testing.assert_allclose(differences(x, lambda v: loss(v, w, b)), dz, atol=1e-7)
    np.testing.assert_allclose(differences(w, lambda v: loss(x, v, b)), dw, atol=1e-7)
    np.testing.assert_allclose(differences(b, lambda v: loss(x, w, v)), db, atol=1e-7)


# ------------------------------------------------------------------ C ABI
def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^(?:int|int64_t)\s+([a-z]\w*)\s*\(", text, flags=re.M)))


def test_header_and_library_agree(L):
    names = declared()
    assert set(names) == {"layer_norm", "layer_norm_backward", "dropout_add",
                          "dropout_add_layer_norm", "quantize_int8", "layer_norm_quantize_int8",
                          "int8_gemm", "int8_linear", "int8_linear_workspace"}
    assert not [n for n in names if not hasattr(L, n)]
    text = open(HEADER).read()
    assert f"FP8DP_NORM_PARTS {sq.NORM_PARTS}" in text
    assert f"FP8DP_INT8_MAX_K {sq.INT8_MAX_K}" in text


def test_c_refusals(L):
    def refused(rc, word):
        assert rc == -1 and word in L.fp8dp_last_error(), L.fp8dp_last_error()

    nan, inf = float("nan"), float("inf")
    # layer_norm(x, weight, bias, rows, cols, dt, wt, eps, y, mean, rstd, stream)
    ln = lambda x=16, w=16, b=16, r=4, c=8, dt=0, wt=0, eps=1e-5, y=32, m=None, s=None: \
        L.layer_norm(x, w, b, r, c, dt, wt, eps, y, m, s, None)
    refused(ln(x=None), b"non-NULL")
    refused(ln(y=None), b"non-NULL")
    for r, c in ((0, 8), (4, 0), (-1, 8), (1 << 31, 8), (4, (1 << 30) + 1)):
        refused(ln(r=r, c=c), b"rows")
    refused(ln(dt=3), b"type")
    refused(ln(dt=0, wt=1), b"type")
    refused(ln(x=17), b"aligned")
    refused(ln(w=18, wt=2), b"aligned")
    refused(ln(m=18), b"aligned")
    for eps in (-1e-9, nan, inf):
        refused(ln(eps=eps), b"eps")
    # dropout_add(x, residual, rows, cols, dt, p, rng, out, stream)
    da = lambda x=16, r=4, c=8, dt=0, p=0.5, g=16, o=32: L.dropout_add(x, None, r, c, dt, p, g, o,
                                                                       None)
    refused(da(x=None), b"non-NULL")
    refused(da(r=0), b"rows")
    refused(da(dt=-1), b"type")
    for p in (-0.1, 1.5, nan):
        refused(da(p=p), b"p must")
    refused(da(g=None), b"rng")
    refused(da(g=20), b"aligned")
    # dropout_add_layer_norm(x, residual, w, b, rows, cols, dt, wt, p, rng, eps, z, y, mean, rstd, stream)
    dl = lambda p=0.5, g=16, eps=1e-5, z=32, y=64, r=4: L.dropout_add_layer_norm(
        16, 16, 16, 16, r, 8, 0, 0, p, g, eps, z, y, None, None, None)
    refused(dl(z=None), b"non-NULL")
    refused(dl(y=32), b"same buffer")
    refused(dl(g=None), b"rng")
    refused(dl(p=2.0), b"p must")
    refused(dl(eps=-1.0), b"eps")
    refused(dl(r=0), b"rows")
    # layer_norm_backward(dy, z, w, mean, rstd, dz_add, rows, cols, dt, wt, p, rng, dz, dx, dw, db, ws, stream)
    lb = lambda dy=16, z=16, m=16, add=None, r=4, dt=0, wt=0, p=0.0, g=None, dz=32, dx=None, \
        dw=16, db=16, ws=16: L.layer_norm_backward(dy, z, 16, m, 16, add, r, 8, dt, wt, p, g, dz,
                                                  dx, dw, db, ws, None)
    for kw in ({"dy": None}, {"z": None}, {"m": None}, {"dz": None}):
        refused(lb(**kw), b"non-NULL")
    refused(lb(dw=None), b"together")
    refused(lb(ws=None), b"workspace")
    refused(lb(r=0), b"rows")
    refused(lb(wt=1), b"type")
    refused(lb(p=-1.0), b"p must")
    refused(lb(p=0.5, dx=64), b"rng")
    refused(lb(dz=16), b"different")
    refused(lb(dz=32, dx=32), b"different")
    refused(lb(m=18), b"aligned")
    # quantize_int8(x, rows, cols, dt, q, scale, stream)
    refused(L.quantize_int8(16, 4, 8, 0, None, 16, None), b"non-NULL")
    refused(L.quantize_int8(16, 4, 8, 5, 16, 16, None), b"type")
    refused(L.quantize_int8(17, 4, 8, 0, 16, 16, None), b"aligned")
    refused(L.quantize_int8(16, 0, 8, 0, 16, 16, None), b"rows")
    # layer_norm_quantize_int8(x, residual, w, b, rows, cols, dt, wt, eps, z, q, scale, stream)
    lq = lambda res=None, z=None, q=16, eps=1e-5, wt=0: L.layer_norm_quantize_int8(
        16, res, 16, 16, 4, 8, 0, wt, eps, z, q, 16, None)
    refused(lq(q=None), b"non-NULL")
    refused(lq(res=16), b"together")
    refused(lq(z=16), b"together")
    refused(lq(eps=nan), b"eps")
    refused(lq(wt=1), b"type")
    # int8_gemm(a, b, M, N, K, sa, sb, bias, yt, bt, y, workspace, bytes, stream)
    ig = lambda a=16, m=4, n=4, k=16, sa=16, yt=0, bt=0, y=16, ws=None, room=0: L.int8_gemm(
        a, 16, m, n, k, sa, 16, None, yt, bt, y, ws, room, None)
    refused(ig(a=None), b"NULL")
    refused(ig(y=None), b"NULL")
    for kw in ({"m": 0}, {"n": 0}, {"k": 0}, {"m": -5}, {"k": sq.INT8_MAX_K + 1},
               {"m": (1 << 30) + 1}):
        refused(ig(**kw), b"must be")
    refused(ig(yt=9), b"type")
    refused(ig(yt=0, bt=1), b"type")
    refused(ig(ws=8, room=64), b"workspace")
    refused(ig(ws=16, room=-1), b"workspace")
    refused(ig(sa=18), b"aligned")
    refused(ig(y=17), b"aligned")
    # int8_linear(x, w8, w_scale, bias, M, N, K, dt, bt, y, workspace, bytes, stream)
    assert L.int8_linear_workspace(3, 17) == 3 * 32 + 16
    il = lambda ws=16, room=112, k=17: L.int8_linear(16, 16, 16, None, 3, 4, k, 0, 0, 16, ws, room,
                                                     None)
    refused(il(ws=None), b"NULL")
    refused(il(room=111), b"112 bytes")
    refused(il(ws=24), b"workspace")
    refused(il(k=0), b"must be")


# ------------------------------------------------------------------ binding
def test_binding_refusals(L):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    f32, i8 = torch.zeros, lambda *s: torch.zeros(*s, dtype=torch.int8)
    rng = torch.zeros(2, dtype=torch.int64)
    E = sq.Fp8dpError
    x, w = bf(4, 16), bf(16)
    for call, word in (
            (lambda: sq.layer_norm(i8(4, 16), w, w, 1e-5, x), "x: expected bfloat16"),
            (lambda: sq.layer_norm(x, w, w, 1e-5, f32(4, 16)), "y: expected"),
            (lambda: sq.layer_norm(x, w, w, 1e-5, bf(4, 8)), "y: expected"),
            (lambda: sq.layer_norm(x, bf(8), w, 1e-5, bf(4, 16)), "16 values"),
            (lambda: sq.layer_norm(x, w, f32(16), 1e-5, bf(4, 16)), "all"),
            (lambda: sq.layer_norm(x, w.half(), None, 1e-5, bf(4, 16)), "all"),
            (lambda: sq.layer_norm(x, w, w, 1e-5, bf(4, 16), f32(3)), "mean: expected 4"),
            (lambda: sq.layer_norm(x, w, w, 1e-5, bf(4, 16), None, bf(4)), "rstd: expected 4"),
            (lambda: sq.layer_norm(bf(()), None, None, 1e-5, bf(())), "dimension"),
            (lambda: sq.layer_norm(x, w, w, 1e-5, bf(4, 16)), "device tensor"),
            (lambda: sq.layer_norm_backward(bf(4, 8), x, w, f32(4), f32(4), x), "dy: expected"),
            (lambda: sq.layer_norm_backward(x, x, w, f32(4), f32(4), x, f32(16), f32(16), f32(127)),
             "workspace"),
            (lambda: sq.layer_norm_backward(x, x, w, f32(4), f32(4), x, f32(15), f32(16), f32(128)),
             "dweight"),
            (lambda: sq.layer_norm_backward(x, x, w, f32(4), f32(4), x, dz_add=bf(3, 16)),
             "dz_add: expected"),
            (lambda: sq.layer_norm_backward(x, x, w, f32(4), f32(4), x, rng=f32(2)), "rng"),
            (lambda: sq.dropout_add(x, bf(4, 8), 0.1, rng, x), "residual: expected"),
            (lambda: sq.dropout_add(x, None, 0.1, rng.int(), x), "rng"),
            (lambda: sq.dropout_add(x, None, 0.1, rng, x.half()), "out: expected"),
            (lambda: sq.dropout_add_layer_norm(x, None, 0.1, rng, w, w, 1e-5, x, bf(4, 1)),
             "y: expected"),
            (lambda: sq.quantize_int8(x, x, f32(4)), "int8 codes"),
            (lambda: sq.quantize_int8(x, i8(4, 8), f32(4)), "x's shape"),
            (lambda: sq.quantize_int8(x, i8(4, 16), f32(5)), "scale: expected 4"),
            (lambda: sq.layer_norm_quantize_int8(x, w, w, 1e-5, i8(4, 16), f32(4), f32(4, 16), x),
             "residual: expected"),
            (lambda: sq.int8_gemm(x, i8(8, 16), f32(4), f32(8), bf(4, 8)), "a: expected int8"),
            (lambda: sq.int8_gemm(i8(4, 16), i8(8, 15), f32(4), f32(8), bf(4, 8)), "shape"),
            (lambda: sq.int8_gemm(i8(4, 16), i8(8, 16), f32(4), f32(8), bf(3, 8)), "shape"),
            (lambda: sq.int8_gemm(i8(4, 16), i8(8, 16), f32(3), f32(8), bf(4, 8)), "a_scale"),
            (lambda: sq.int8_gemm(i8(4, 16), i8(8, 16), f32(4), f32(9), bf(4, 8)), "weight scale"),
            (lambda: sq.int8_gemm(i8(4, 16), i8(8, 16), f32(4), f32(8), bf(4, 8), bf(9)), "bias"),
            (lambda: sq.int8_linear(x, i8(8, 16), f32(8), f32(4, 8), i8(1 << 12)), "x's type"),
    ):
        with pytest.raises(E, match=word):
            call()
