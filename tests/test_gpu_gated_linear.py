"""The gated linear layer and its backward pass on the GPU, against their 64-bit definitions
(oracle/gated.py).

Tolerances, from the arithmetic.  H is half a step of the type relative to a value, U = 2^-24.  A sum over K
goes through matrix instructions that add 16 or 32 products each; a product meets at most 32 roundings
inside its instruction, K / 16 in the accumulator, and 16 where partial sums are joined, and a
matrix instruction may truncate, which is 2 U.  So a sum is off by at most
E = (K / 16 + 48) 2 U times the sum of magnitudes.  f and its derivative come from exp, a reciprocal and
erfc of a few units in the last place, whose arguments are off by a few U themselves, which exp turns
into that many U times the argument (below 1.6 |g| + 0.08 |g|^3): F = (32 + 8 |g| + 4 g^2 + |g|^3) U
relative to f, and (1 + |g|) F for the derivative.
"""
import numpy as np
import pytest
import torch

import oracle.gated as OG
import scaled_quantization_amd as sq
from gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F16 = torch.bfloat16, torch.float16
ACT = {name: i for i, name in enumerate(OG.ACTS)}


def half(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half the smallest step of type t."""
    return {BF16: 2.0 ** -134, F16: 2.0 ** -25}[t]


def draw(shape, t, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(t)


def f64(x):
    return x.cpu().double().numpy()


def close(got, ref, tol, what):
    got = f64(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {ref[bad][0]}, allowed {tol[bad][0]}")


def scratch(n, value=255):
    return torch.full((max(n, 16),), value, dtype=torch.uint8, device=DEV)


def fn_error(g):
    g = np.abs(g)
    return (32 + 8 * g + 4 * g * g + g ** 3) * U


def check_forward(x, wg, wu, act, h, gate, up, t, what):
    x, wg, wu = f64(x), f64(wg), f64(wu)
    ref, g, u = OG.gated_linear(x, wg, wu, act)
    e = (x.shape[1] / 16 + 48) * 2 * U
    eg, eu = e * (np.abs(x) @ np.abs(wg).T), e * (np.abs(x) @ np.abs(wu).T)
    if gate is not None:
        close(gate, g, eg + half(t) * (np.abs(g) + eg) + tiny(t), what + " gate")
        close(up, u, eu + half(t) * (np.abs(u) + eu) + tiny(t), what + " up")
    slope = 2 * (np.abs(g) + eg) if act == "relu2" else 1.2     # |f'| of the others is below
    f = np.abs(OG.activation(g, act)[0])
    off = slope * eg * (np.abs(u) + eu) + f * eu + fn_error(g) * f * (np.abs(u) + eu)
    close(h, ref, off + half(t) * (np.abs(ref) + off) + tiny(t), what + " h")


def forward(M, N, K, t, act, train, seed=0, workspace=True):
    x, wg, wu = draw((M, K), t, seed), draw((N, K), t, seed + 1, K ** -0.5), draw((N, K), t, seed + 2, K ** -0.5)
    h = torch.full((M, N), float("nan"), dtype=t, device=DEV)
    gate, up = (torch.full_like(h, float("nan")) for _ in range(2)) if train else (None, None)
    ws = scratch(sq.gated_linear_workspace(M, N, K)) if workspace else None
    sq.gated_linear(x.to(DEV), wg.to(DEV), wu.to(DEV), ACT[act], h, gate, up, ws)
    check_forward(x, wg, wu, act, h, gate, up, t, f"{M}x{N}x{K}")
    return h


# every kernel, both sides of each change between them, cut tiles in every dimension, one of each
SHAPES = [(1, 1, 1), (1, 16, 8), (1, 2048, 768), (3, 17, 7), (16, 100, 129), (17, 33, 1000), (33, 64, 256),
          (48, 65, 1001), (64, 31, 4104), (65, 64, 64), (65, 40, 72), (100, 129, 1), (128, 128, 4096),
          (129, 63, 513), (300, 1000, 80), (257, 300, 1001), (513, 4112, 192), (1, 5, 20000), (2000, 8, 24)]


@pytest.mark.parametrize("t", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward_shapes(shape, t):
    forward(*shape, t, "silu", True)


@pytest.mark.parametrize("M", [1, 40, 200])
@pytest.mark.parametrize("act", OG.ACTS)
def test_forward_activations(act, M):
    forward(M, 72, 136, F16, act, M == 40)
    forward(M, 72, 136, BF16, act, M != 40)


@pytest.mark.parametrize("M", [1, 16, 17, 32, 33, 48, 49, 64])
def test_forward_few_tokens_and_many_weights(M):
    # rings of weights: fewer groups of channels than workgroups, more of them, stages that K cuts
    forward(M, 1100, 4104, BF16, "silu", M % 2 == 0)
    forward(M, 4500, 1000, F16, "gelu_tanh", M % 2 == 1)
    forward(M, 4112, 1024, BF16, "relu", False)
    forward(M, 16400, 264, F16, "silu", False)


def test_forward_large_tiles_and_no_workspace():
    forward(2048, 4096, 128, BF16, "silu", True)
    forward(2111, 4200, 72, F16, "gelu_tanh", False)
    forward(130, 128, 4096, BF16, "silu", False, workspace=False)


def test_workspace_form_is_the_same_up_to_rounding():
    # split and not split: both within the bound of the same reference, and the workspace is used
    assert sq.gated_linear_workspace(130, 128, 4096) > 0
    a, b = (forward(130, 128, 4096, BF16, "silu", False, workspace=w) for w in (True, False))
    assert (a.float() - b.float()).abs().max() <= 2 ** -7 * a.float().abs().max()


@pytest.mark.parametrize("M", [5, 100, 300])
@pytest.mark.parametrize("offset", [1, 4])
def test_forward_at_any_alignment(M, offset):
    # operands and outputs that start at any element
    N, K, t = 72, 128, BF16
    ins = [draw((M, K), t, 3), draw((N, K), t, 4, 0.1), draw((N, K), t, 5, 0.1)]
    dev = []
    for v in ins:
        room = torch.empty(v.numel() + offset, dtype=t, device=DEV)
        room[offset:] = v.reshape(-1).to(DEV)
        dev.append(room[offset:].view(v.shape))
    outs = []
    for _ in range(3):
        room = torch.full((M * N + 2 * offset,), 7.0, dtype=t, device=DEV)
        outs.append((room, room[offset:-offset].view(M, N)))
    sq.gated_linear(*dev, sq.GATE_SILU, *(o for _, o in outs), scratch(sq.gated_linear_workspace(M, N, K)))
    check_forward(*ins, "silu", *(o for _, o in outs), t, "offset")
    for room, _ in outs:
        assert (room[:offset] == 7).all() and (room[-offset:] == 7).all()


@pytest.mark.parametrize("M", [7, 140])
def test_rows_that_are_not_finite_touch_no_other(M):
    N, K = 40, 72
    x, wg, wu = draw((M, K), BF16, 1), draw((N, K), BF16, 2, 0.1), draw((N, K), BF16, 3, 0.1)
    x[2, 5], x[3, 71] = float("nan"), float("inf")
    h = torch.empty((M, N), dtype=BF16, device=DEV)
    sq.gated_linear(x.to(DEV), wg.to(DEV), wu.to(DEV), sq.GATE_SILU, h, workspace=scratch(
        sq.gated_linear_workspace(M, N, K)))
    assert not torch.isfinite(h[2]).any()
    keep = [i for i in range(M) if i not in (2, 3)]
    assert torch.isfinite(h[keep]).all()
    # a weight row that is not finite stays in its channel
    x = draw((M, K), BF16, 1)
    wu[39, 0] = float("inf")
    sq.gated_linear(x.to(DEV), wg.to(DEV), wu.to(DEV), sq.GATE_SILU, h, workspace=scratch(
        sq.gated_linear_workspace(M, N, K)))
    assert torch.isfinite(h[:, :39]).all() and not torch.isfinite(h[:, 39]).any()


# ------------------------------------------------------------------ backward
def check_backward(dh, gate, up, x, wg, wu, act, dx, dwg, dwu, t, what):
    dh, g, u, x, wg, wu = (f64(v) for v in (dh, gate, up, x, wg, wu))
    f, slope = OG.activation(g, act)
    rdx, rg, ru = OG.gated_linear_backward(dh, g, u, x, wg, wu, act)
    dg, du = np.abs(dh * u * slope), np.abs(dh * f)
    fe = fn_error(g)
    # dg and du as the products see them: the functions' errors, three products, one rounding to t
    off_g = np.abs(dh * u) * (1 + np.abs(g)) * fe * (2 if act != "relu2" else 2 + 2 * np.abs(g)) + 4 * U * dg
    off_u = du * (fe + 4 * U)
    off_g, off_u = (o + half(t) * (d + o) + tiny(t) for o, d in ((off_g, dg), (off_u, du)))

    def bound(terms, ref, n):
        e = (n / 16 + 48) * 2 * U
        off = sum(o @ m + e * ((d + o) @ m) for o, d, m in terms)
        return off + half(t) * (np.abs(ref) + off) + tiny(t)

    if dx is not None:
        terms = ((off_g, dg, np.abs(wg)), (off_u, du, np.abs(wu)))
        close(dx, rdx, bound(terms, rdx, 2 * g.shape[1] + 128), what + " dx")
    if dwg is not None:
        n = g.shape[0] + 64
        close(dwg, rg, bound(((off_g.T, dg.T, np.abs(x)),), rg, n), what + " dw_gate")
        close(dwu, ru, bound(((off_u.T, du.T, np.abs(x)),), ru, n), what + " dw_up")


def backward_inputs(M, N, K, t, seed=0):
    x, wg, wu = draw((M, K), t, seed), draw((N, K), t, seed + 1, K ** -0.5), draw((N, K), t, seed + 2, K ** -0.5)
    return draw((M, N), t, seed + 3, 0.1), draw((M, N), t, seed + 4, 1.5), draw((M, N), t, seed + 5), x, wg, wu


def backward(M, N, K, t, act, want_dx=True, want_dw=True, seed=0):
    ins = backward_inputs(M, N, K, t, seed)
    dx = torch.full((M, K), float("nan"), dtype=t, device=DEV) if want_dx else None
    dwg, dwu = (torch.full((N, K), float("nan"), dtype=t, device=DEV) if want_dw else None for _ in range(2))
    ws = scratch(sq.gated_linear_backward_workspace(M, N, K))   # (all bytes 255: NaN in every type)
    sq.gated_linear_backward(*(v.to(DEV) for v in ins), ACT[act], ws, dx, dwg, dwu)
    check_backward(*ins, act, dx, dwg, dwu, t, f"{M}x{N}x{K}")


@pytest.mark.parametrize("t", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward_shapes(shape, t):
    backward(*shape, t, "silu")


@pytest.mark.parametrize("act", OG.ACTS)
def test_backward_activations(act):
    backward(70, 72, 136, F16, act)
    backward(33, 40, 64, BF16, act)


def test_backward_large_tiles_and_parts():
    backward(4096, 512, 1024, BF16, "silu")     # 256 x 256 tiles
    backward(2048, 1000, 776, F16, "silu")
    backward(8192, 64, 64, BF16, "silu")        # the weights' gradients in ranges of the tokens
    backward(260, 96, 72, BF16, "silu", want_dw=False)
    backward(260, 96, 72, BF16, "silu", want_dx=False)


def test_backward_against_differences():
    # d sum(h v) of the kernel's own forward pass in one direction of each input: the difference of h over
    # 2 s directions is the gradient's product with the direction up to s^2 and the roundings of h, 2^-11 a value
    M, N, K, t = 40, 24, 32, F16
    dh, _, _, x, wg, wu = backward_inputs(M, N, K, t, 7)
    args = [v.to(DEV) for v in (x, wg, wu)]
    gate, up, h = (torch.empty((M, N), dtype=t, device=DEV) for _ in range(3))
    sq.gated_linear(*args, sq.GATE_SILU, h, gate, up)
    dx, dwg, dwu = torch.empty_like(args[0]), torch.empty_like(args[1]), torch.empty_like(args[1])
    sq.gated_linear_backward(dh.to(DEV), gate, up, *args, sq.GATE_SILU,
                             scratch(sq.gated_linear_backward_workspace(M, N, K)), dx, dwg, dwu)
    step = 2.0 ** -3
    for i, grad in enumerate((dx, dwg, dwu)):
        # a direction of +-1 or 0 along the gradient's signs: x + step d is exact enough in float64 only,
        # so the difference is the definition's, and the kernel's gradient is held to it
        d = np.sign(f64(grad)) * (np.abs(f64(grad)) > np.median(np.abs(f64(grad))))
        ends = []
        for s in (step, -step):
            ins = [f64(v) for v in (x, wg, wu)]
            ins[i] = ins[i] + s * 2 ** -6 * d
            ends.append((OG.gated_linear(*ins, "silu")[0] * f64(dh)).sum())
        diff = (ends[0] - ends[1]) / (2 * step * 2 ** -6)
        got = (f64(grad) * d).sum()
        # central differences are off by the third derivative (the steps move g by 2^-9 sum |w| < 2^-5:
        # its square by 6 is below 2e-4 of the whole); the gradient by five roundings to 16 bits (gate, up, dg or
        # du, itself, and f'' times gate's), all to one side at worst
        assert abs(got - diff) <= (5 * half(t) + 2e-4) * np.abs(f64(grad) * d).sum()


def test_same_call_same_bits():
    ins = [v.to(DEV) for v in backward_inputs(1000, 136, 264, BF16)]
    ws = scratch(sq.gated_linear_backward_workspace(1000, 136, 264))
    outs = []
    for fill in (255, 0, 17):
        ws.fill_(fill)
        o = [torch.empty_like(ins[3]), torch.empty_like(ins[4]), torch.empty_like(ins[4])]
        sq.gated_linear_backward(*ins, sq.GATE_SILU, ws, *o)
        outs.append(o)
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


@pytest.mark.parametrize("M", [20, 500])
def test_captured_and_replayed(M):
    # one graph of forward and backward, replayed on new inputs, with eager work between
    N, K, t = 136, 264, BF16
    dh, gate, up, x, wg, wu = (v.to(DEV) for v in backward_inputs(M, N, K, t))
    h, dx, dwg, dwu = torch.empty_like(gate), torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wg)
    ws = scratch(max(sq.gated_linear_workspace(M, N, K), sq.gated_linear_backward_workspace(M, N, K)))

    def step():
        sq.gated_linear(x, wg, wu, sq.GATE_SILU, h, gate, up, ws)
        sq.gated_linear_backward(dh, gate, up, x, wg, wu, sq.GATE_SILU, ws, dx, dwg, dwu)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        x.copy_(draw((M, K), t, 100 + seed))
        dh.copy_(draw((M, N), t, 200 + seed, 0.1))
        for v in (h, gate, up, dx, dwg, dwu):
            v.fill_(float("nan"))
        graph.replay()
        got = [v.clone() for v in (h, gate, up, dx, dwg, dwu)]
        torch.cuda.synchronize()
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (h, gate, up, dx, dwg, dwu)))


def test_on_another_stream():
    M, N, K = 300, 72, 128
    x, wg, wu = (v.to(DEV) for v in (draw((M, K), BF16, 1), draw((N, K), BF16, 2, 0.1), draw((N, K), BF16, 3, 0.1)))
    h = torch.empty((M, N), dtype=BF16, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = scratch(sq.gated_linear_workspace(M, N, K))
    s.wait_stream(torch.cuda.current_stream())
    sq.gated_linear(x, wg, wu, sq.GATE_SILU, h, workspace=ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    check_forward(x, wg, wu, "silu", h, None, None, BF16, "stream")
