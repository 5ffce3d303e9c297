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
