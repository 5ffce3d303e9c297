"""The kernels of the gated linear layer's large products, each at sizes that reach it (tests/gated_shapes.py), against
the definition in 64 bits.

Tolerances as in tests/test_gpu_gated_linear.py: a sum over K is off by at most E = (K / 16 + 48) 2 U times the sum of
magnitudes, U = 2^-24; the functions by F = (32 + 8 |g| + 4 g^2 + |g|^3) U; H is half a step of the type.  The matrices of
magnitudes are formed in binary32, which is off by far less than the bounds are wide, and taken 1.01 times.
"""
import pytest
import torch

import gated_shapes as S
import scaled_quantization_amd as sq
from gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F16 = torch.bfloat16, torch.float16
TINY = {BF16: 2.0 ** -134, F16: 2.0 ** -25}


def half(t):
    return torch.finfo(t).eps / 2


def draws(t, seed, *shapes):
    """Normal values, shapes with their standard deviation."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [(torch.randn(s, generator=g, device=DEV) * std).to(t) for s, std in shapes]


def product(a, b):
    """a b^T in 64 bits, in pieces of a."""
    b = b.double().t().contiguous()
    return torch.cat([torch.matmul(v.double(), b) for v in a.split(2048)])


def sizes(a, b):
    return torch.matmul(a.float().abs(), b.float().abs().t().contiguous()).double() * 1.01


def silu(g):
    p = torch.sigmoid(g)
    return g * p, p * (1 + g * (1 - p))


def fn_error(g):
    g = g.abs()
    return (32 + 8 * g + 4 * g * g + g ** 3) * U


def close(got, ref, tol, what):
    bad = ~((got.double() - ref).abs() <= tol)
    n = int(bad.sum())
    assert n == 0, (f"{what}: {n} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}: {got[bad][0].item()} for "
                    f"{ref[bad][0].item()}, allowed {tol[bad][0].item()}")


def scratch(n):
    return torch.full((max(n, 16),), 255, dtype=torch.uint8, device=DEV)


def nan(*shape, t):
    return torch.full(shape, float("nan"), dtype=t, device=DEV)


def forward(M, N, K, t, train):
    x, wg, wu = draws(t, M, ((M, K), 1.0), ((N, K), K ** -0.5), ((N, K), K ** -0.5))
    h, gate, up = nan(M, N, t=t), *((nan(M, N, t=t), nan(M, N, t=t)) if train else (None, None))
    sq.gated_linear(x, wg, wu, sq.GATE_SILU, h, gate, up, scratch(sq.gated_linear_workspace(M, N, K)))
    g, u = product(x, wg), product(x, wu)
    e = (K / 16 + 48) * 2 * U
    eg, eu = e * sizes(x, wg), e * sizes(x, wu)
    if train:
        close(gate, g, eg + half(t) * (g.abs() + eg) + TINY[t], "gate")
        close(up, u, eu + half(t) * (u.abs() + eu) + TINY[t], "up")
    f = silu(g)[0]
    off = 1.2 * eg * (u.abs() + eu) + f.abs() * eu + fn_error(g) * f.abs() * (u.abs() + eu)
    close(h, f * u, off + half(t) * ((f * u).abs() + off) + TINY[t], "h")


def shape_id(s):
    return "x".join(map(str, s))


@pytest.mark.parametrize("train", [False, True], ids=["h", "training"])
@pytest.mark.parametrize("shape", [*S.FORWARD.values(), S.PADDED["forward"]], ids=shape_id)
def test_forward(shape, train):
    forward(*shape, BF16 if train else F16, train)


def backward(M, N, K, t, which):
    dh, gate, up, x, wg, wu = draws(t, M + 1, ((M, N), 0.1), ((M, N), 1.5), ((M, N), 1.0), ((M, K), 1.0),
                                    ((N, K), K ** -0.5), ((N, K), K ** -0.5))
    dx = nan(M, K, t=t) if which == "dx" else None
    dw = [nan(N, K, t=t) if which == "dw" else None for _ in range(2)]
    sq.gated_linear_backward(dh, gate, up, x, wg, wu, sq.GATE_SILU,
                             scratch(sq.gated_linear_backward_workspace(M, N, K)), dx, *dw)
    d, g, u = dh.double(), gate.double(), up.double()
    f, slope = silu(g)
    fe = fn_error(g)
    # each term with its error: the functions', three products, one rounding to t
    dg, du = d * u * slope, d * f
    off_g = (d * u).abs() * (1 + g.abs()) * fe * 2 + 4 * U * dg.abs()
    off_u = du.abs() * (fe + 4 * U)
    off_g, off_u = (o + half(t) * (v.abs() + o) + TINY[t] for o, v in ((off_g, dg), (off_u, du)))

    def bound(terms, ref, n):
        e = (n / 16 + 48) * 2 * U
        off = sum(sizes(o + e * (v.abs() + o), w) for o, v, w in terms)
        return off + half(t) * (ref.abs() + off) + TINY[t]

    if dx is not None:
        wgt, wut = wg.t().contiguous(), wu.t().contiguous()
        ref = product(dg, wgt) + product(du, wut)
        close(dx, ref, bound(((off_g, dg, wgt), (off_u, du, wut)), ref, 2 * N + 128), "dx")
    else:
        xt = x.t().contiguous()
        for got, v, o, what in ((dw[0], dg, off_g, "dw_gate"), (dw[1], du, off_u, "dw_up")):
            v, o = v.t().contiguous(), o.t().contiguous()
            ref = product(v, xt)
            close(got, ref, bound(((o, v, xt),), ref, M + 64), what)


@pytest.mark.parametrize("t", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", [*S.DX.values(), S.PADDED["dx"]], ids=shape_id)
def test_gradient_of_x(shape, t):
    backward(*shape, t, "dx")


@pytest.mark.parametrize("t", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", [*S.DW.values(), S.PADDED["dw"]], ids=shape_id)
def test_gradients_of_the_weights(shape, t):
    backward(*shape, t, "dw")
