"""The gated linear layer's gradient where an activation has saturated, against its 64-bit definition
(oracle/gated.py).

With one token dw_gate[n, k] is dg[n] x[k] alone, so every error is relative to the derivative itself.  Tolerance: the
functions' errors are those of tests/test_gpu_gated_linear.py, F = (32 + 8 |g| + 4 g^2 + |g|^3) 2^-24 relative, for a
derivative that is a product or a sum without cancelling twice that, three products, and one rounding to the type each of
dg and the output.  A sigmoid or exponential below binary32's smallest normal, 2^-126, may be 0.  A derivative has it times |g| at most, that
of the tanh form times |g| 2 sqrt(2 / pi) (1 + 0.134145 g^2), the derivative of its argument (235 at g = -10.06, where the
sigmoid is e^-88.3 < 2^-126 and the derivative 6.6e-37 = 56 2^-126); dh, up and x, below 1.5 each, come on top.
"""
import numpy as np
import pytest
import torch

import oracle.gated as OG
import scaled_quantization_amd as sq
from gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = torch.bfloat16


def f64(x):
    return x.cpu().double().numpy()


def backward(dh, gate, up, x, wg, wu, act, dx=False):
    M, N, K = *gate.shape, x.shape[1]
    ws = torch.full((sq.gated_linear_backward_workspace(M, N, K),), 255, dtype=torch.uint8, device=DEV)
    out = [torch.full_like(v, float("nan"), device=DEV) for v in ((x,) if dx else ()) + (wg, wu)]
    sq.gated_linear_backward(*(v.to(DEV) for v in (dh, gate, up, x, wg, wu)), OG.ACTS.index(act), ws,
                             *(out if dx else [None] + out))
    return out


@pytest.mark.parametrize("act", ["sigmoid", "silu", "gelu", "gelu_tanh"])
def test_saturated_gates(act):
    # -30 .. 30 without the roots of the derivatives near -1
    g = torch.cat([torch.linspace(-30, -3, 200), torch.linspace(3, 30, 200)])
    if act == "sigmoid":
        g = torch.cat([g, torch.linspace(-3, 3, 100)])
    g = g.to(BF16)[None]
    gen = torch.Generator().manual_seed(1)
    rand = lambda *s: (0.5 + torch.rand(s, generator=gen)).to(BF16)
    N, K = g.shape[1], 24
    dh, up, x, w = rand(1, N), rand(1, N), rand(1, K), rand(N, K)
    dwg, dwu = (f64(v) for v in backward(dh, g, up, x, w, w, act))
    _, rg, ru = OG.gated_linear_backward(*(f64(v) for v in (dh, g, up, x, w, w)), act)
    a = np.abs(f64(g)).T
    fe = (32 + 8 * a + 4 * a * a + a ** 3) * U
    low = 4 * (1 + a * (1.6 * (1 + 0.1342 * a * a) if act == "gelu_tanh" else 1)) * 2.0 ** -126
    step = 2 * 2.0 ** -8 + 2.0 ** -16
    assert (np.abs(dwg - rg) <= np.abs(rg) * (2 * fe + 4 * U + step) + low).all()
    assert (np.abs(dwu - ru) <= np.abs(ru) * (fe + 4 * U + step) + low).all()


# ------------------------------------------------------------------ float16's range
# The largest finite |dg| or |du| of a call is m.  dg and du keep half a step of float16 relative to each, or in absolute
# terms half its smallest step: 2^-25, or, where m leaves [2^-6, 2^15] and all share a power of two that brings it to
# [2^14, 2^15), 2^-25 m 2^-14.
F16 = torch.float16


def scaled_inputs(M, N, K, power, seed=0):
    """Magnitudes of about 2^power for dg and du, and weights and tokens that bring the gradients back to 1."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s, to: (torch.randn(s, generator=gen) * to).to(F16)
    each, back = 2.0 ** (power / 2), 2.0 ** -max(power, 0)
    return (rand(M, N, to=each), rand(M, N, to=1.5), rand(M, N, to=each), rand(M, K, to=back * M ** -0.5 * 8),
            rand(N, K, to=back * N ** -0.5 * 8), rand(N, K, to=back * N ** -0.5 * 8))


def check(ins, act, dx, dwg, dwu, rows=slice(None)):
    dh, g, u, x, wg, wu = (f64(v) for v in ins)
    f, slope = OG.activation(g, act)
    dg, du = np.abs(dh * u * slope), np.abs(dh * f)
    a = np.abs(g)
    fe = (32 + 8 * a + 4 * a * a + a ** 3) * U
    m = max(dg[np.isfinite(dg)].max(), du[np.isfinite(du)].max())
    least = 2.0 ** -25 if 2.0 ** -6 <= m <= 2.0 ** 15 else m * 2.0 ** -39
    # (the derivative's error relative to 1 + |g|, as it may cancel)
    off_g = np.abs(dh * u) * (1 + a) * fe * 2 + dg * 4 * U
    off_u = du * (fe + 4 * U)
    off_g, off_u = (o + 2.0 ** -11 * (d + o) + least for o, d in ((off_g, dg), (off_u, du)))

    def close(got, terms, ref, n):
        e = (n / 16 + 48) * 2 * U
        off = sum(o @ v + e * ((d + o) @ v) for o, d, v in terms)
        tol = off + 2.0 ** -11 * (np.abs(ref) + off) + 2.0 ** -25
        got = f64(got)
        bad = ~(np.abs(got - ref) <= tol)[rows]
        assert not bad.any(), (m, bad.sum(), got[rows][bad][0], ref[rows][bad][0], tol[rows][bad][0])

    rdx, rg, ru = OG.gated_linear_backward(dh, g, u, x, wg, wu, act)
    close(dx, ((off_g, dg, np.abs(wg)), (off_u, du, np.abs(wu))), rdx, 2 * g.shape[1] + 128)
    if dwg is not None:
        close(dwg, ((off_g.T, dg.T, np.abs(x)),), rg, g.shape[0] + 64)
        close(dwu, ((off_u.T, du.T, np.abs(x)),), ru, g.shape[0] + 64)


# aligned, K in ranges with a join, copied to aligned rows, at any alignment, one token
@pytest.mark.parametrize("shape", [(100, 64, 64), (8192, 64, 64), (300, 260, 301), (70, 40, 33), (1, 200, 72)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("power", [20, 15, 12, 3, -4, -8, -14, -22])
def test_gradient_beyond_float16(shape, power):
    ins = scaled_inputs(*shape, power)
    check(ins, "silu", *backward(*ins, "silu", dx=True))


def test_gradient_of_zeros_and_of_tokens_that_are_not_finite():
    ins = scaled_inputs(90, 64, 72, 18)
    zero = [torch.zeros_like(ins[0]), *ins[1:]]
    assert all((v == 0).all() for v in backward(*zero, "silu", dx=True))
    ins[0][7, 3], ins[2][50, 9] = float("inf"), float("nan")
    dx, dwg, dwu = backward(*ins, "silu", dx=True)
    keep = [i for i in range(90) if i not in (7, 50)]
    with np.errstate(invalid="ignore"):
        check(ins, "silu", dx, None, None, keep)
    assert not torch.isfinite(dx[[7, 50]]).any()
    assert torch.isfinite(dwg[:3]).all() and not torch.isfinite(dwg[3]).any() and torch.isfinite(dwu[4:]).all()


def test_captured_gradient_follows_the_range():
    M, N, K = 300, 136, 72
    dh, gate, up, x, wg, wu = (v.to(DEV) for v in scaled_inputs(M, N, K, 3))
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wg)
    ws = torch.empty(sq.gated_linear_backward_workspace(M, N, K), dtype=torch.uint8, device=DEV)
    step = lambda: sq.gated_linear_backward(dh, gate, up, x, wg, wu, sq.GATE_SILU, ws, dx, dwg, dwu)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for power in (18, 2, -20, 18):
        ins = scaled_inputs(M, N, K, power, power + 50)
        for to, v in zip((dh, gate, up, x, wg, wu), ins):
            to.copy_(v)
        ws.fill_(255)
        graph.replay()
        got = [v.clone() for v in (dx, dwg, dwu)]
        torch.cuda.synchronize()
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (dx, dwg, dwu)))
        check(ins, "silu", *got)
