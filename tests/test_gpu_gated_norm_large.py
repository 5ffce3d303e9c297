"""The gradient of the block norm where a workgroup walks many rows, streams are read past the caches, or rows are on
either side of the limit of a kernel, against the definition in 64 bits.

Tolerances as in tests/test_gpu_gated_norm.py: U = 2^-24 an operation, S = 160 U for a row's sum, half a step of the
type for an output; a sum over rows adds (2 * 64 + 80) U of the sum of magnitudes: up to 64 rows in sequence, as many of
these sums, 4 waves, 1024 partial sums in 32 and 32 steps (where a workgroup walks more than 64 rows of a width that
is in the workspace, what its additions round off is kept).
"""
import pytest
import torch

import scaled_quantization_amd as sq
from gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
S = 160 * U
ROWS = (2 * 64 + 80) * U
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
A, B, EPS = 1.25, -0.75, 1e-5
CACHE = 256 << 20     # bytes of all tensors from which on they are read past the caches


def half(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return {BF16: 2.0 ** -134, F16: 2.0 ** -25, F32: 2.0 ** -150}[t]


def close(got, ref, tol, what):
    bad = ~((got.double() - ref).abs() <= tol)
    n = int(bad.sum())
    assert n == 0, (f"{what}: {n} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}: {got[bad][0].item()} for "
                    f"{ref[bad][0].item()}, allowed {tol[bad][0].item()}")


def inputs(rows, cols, t, kind):
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    rand = lambda *s, std=1.0, mean=0.0: (torch.randn(s, generator=g, device=DEV) * std + mean).to(t)
    x, z, dy, add = rand(rows, cols, std=1.5, mean=0.25), rand(rows, cols, std=2.0), rand(rows, cols), rand(rows, cols)
    post, pre = rand(cols, std=0.3, mean=1.0), rand(cols, std=0.3, mean=1.0)
    gate = rand(*((rows, cols) if kind == "token" else (cols,)), std=0.2, mean=0.5)
    r1, r2 = (torch.cat([torch.rsqrt(p.double().square().mean(1) + EPS) for p in v.split(2048)]).float() for v in (x, z))
    return dy, add, x, z, post, gate, pre, r1, r2


def run(ins, kind, over=(None, None, None)):
    """over: which of the inputs dresidual, dx and a gate's gradient per token take the place of."""
    dy, add, x, z, post, gate, pre, r1, r2 = ins
    rows, cols = x.shape
    place = {"dy": dy.clone(), "add": add.clone()}
    buffers = [place[o] if o else torch.full_like(x, float("nan")) for o in over]
    if kind != "token":
        buffers[2] = torch.full((cols,), float("nan"), device=DEV)
    sums = [torch.full((cols,), float("nan"), device=DEV) for _ in range(2)]
    ws = torch.full((2 * min(rows, sq.NORM_PARTS) * cols,), float("nan"), device=DEV)
    sq.block_norm_backward(place["dy"], place["add"], x, z, post, gate, pre, r1, r2, *buffers, *sums, ws, A, B)
    return [*buffers, *sums]


def check(ins, kind, out, what):
    dy, add, x, z, post, gate, pre, r1, r2 = ins
    t, (rows, cols) = x.dtype, x.shape
    w, p = post.double(), pre.double()
    names = ("dgate", "dpost", "dpre")
    total, wide = ({n: torch.zeros(cols, dtype=torch.float64, device=DEV) for n in names} for _ in range(2))
    for at in range(0, rows, 2048):
        s = slice(at, at + 2048)
        d, a, xh, zh = (v[s].double() for v in (dy, add, x, z))
        q1, q2 = r1[s].double()[:, None], r2[s].double()[:, None]
        g = gate[s].double() if kind == "token" else gate.double()
        xh, zh, c = xh * q1, zh * q2, d * p
        dz = a + q2 * (c - zh * (c * zh).mean(1, keepdim=True))
        e = B * g * dz
        q = e * w
        dx = q1 * (q - xh * (q * xh).mean(1, keepdim=True))
        # magnitudes, and how far each step may be off
        m = (c * zh).abs().mean(1, keepdim=True)
        mz = a.abs() + q2 * (c.abs() + zh.abs() * m)
        off = 12 * U * mz + q2 * zh.abs() * m * (S + 8 * U)
        gw = (B * g * w).abs()
        me, eo = mz * gw, off * gw + 6 * U * mz * gw
        mm = (me * xh.abs()).mean(1, keepdim=True)
        m_off = (eo * xh.abs()).mean(1, keepdim=True) + mm * (S + 4 * U)
        dxo = q1 * (eo + 4 * U * me + xh.abs() * (m_off + 6 * U * mm))
        ref = A * dz
        close(out[0][s], ref, A * off + half(t) * (ref.abs() + A * off) + 2 * U * ref.abs() + tiny(t), what + " dresidual")
        close(out[1][s], dx, dxo + half(t) * (dx.abs() + dxo) + tiny(t), what + " dx")
        dg, go = B * dz * xh * w, (B * w * xh).abs() * (off + 8 * U * mz)
        if kind == "token":
            close(out[2][s], dg, go + half(t) * (dg.abs() + go) + tiny(t), what + " dgate")
        bg = (B * g * xh).abs()
        for n, v, o in (("dgate", dg, go + ROWS * (B * w * xh).abs() * mz), ("dpost", e * xh, bg * (off + (8 * U + ROWS) * mz)),
                        ("dpre", d * zh, (ROWS + 4 * U) * (d * zh).abs())):
            total[n] += v.sum(0)
            wide[n] += o.sum(0)
    for n, got in zip(names, out[2:]):
        if n != "dgate" or kind != "token":
            close(got, total[n], wide[n] + 8 * U * total[n].abs(), what + " " + n)


# rows of the kernel that reads a row again by each step: a workgroup each, and several
@pytest.mark.parametrize("rows, cols", [(1023, 16385), (1024, 16385), (1300, 20001), (3000, 7), (1025, 1), (5000, 3)])
def test_rows_in_steps(rows, cols):
    for t, kind in ((BF16, "token"), (F32, "channel")):
        ins = inputs(rows, cols, t, kind)
        check(ins, kind, run(ins, kind), f"{rows}x{cols} {kind}")


def test_rows_in_steps_in_place():
    ins = inputs(1100, 16387, BF16, "token")
    want = run(ins, "token")
    for over in (("dy", "add", None), ("add", None, "dy")):
        assert all(torch.equal(a, b) for a, b in zip(run(ins, "token", over), want)), over


# every width of threads and registers, cut, from more memory than the caches hold
@pytest.mark.parametrize("t", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cols", [101, 603, 1999, 4095, 8191, 8195, 16381])
def test_streams(cols, t):
    size = 2 if t == BF16 else 4
    for kind, tensors in (("token", 8), ("channel", 6)):
        rows = CACHE // (cols * tensors * size) + 3
        ins = inputs(rows, cols, t, kind)
        out = run(ins, kind)
        check(ins, kind, out, f"{rows}x{cols} {kind}")
        assert all(torch.equal(a, b) for a, b in zip(run(ins, kind, ("dy", "add", None)), out))


@pytest.mark.parametrize("over", [0, 1])
def test_either_side_of_the_row_limit(over):
    # 64 rows for each compute unit, and one more: one pass, and a kernel that reads a row again by each step
    rows = 64 * torch.cuda.get_device_properties(0).multi_processor_count + over
    ins = inputs(rows, 8203, BF16, "channel")
    check(ins, "channel", run(ins, "channel"), f"{rows} rows")


@pytest.mark.parametrize("cols", [2050, 4098, 8194, 8195, 8199, 9001])
def test_cut_vectors_of_another_wave_in_place(cols):
    # without dy no sum over the row comes before the first output; the last vector, cut, is read as the row's
    # last 8 elements, of which other waves write the first ones
    dy, add, x, z, post, gate, pre, r1, r2 = inputs(300, cols, BF16, "token")
    outs = []
    for place in (False, True):
        a = add.clone()
        out = [a if place else torch.empty_like(a), torch.empty_like(a), torch.empty_like(a)]
        sums = torch.empty(cols, device=DEV)
        ws = torch.empty(2 * 300 * cols, device=DEV)
        sq.block_norm_backward(None, a, x, None, post, gate, None, r1, None, *out, sums, None, ws, A, B)
        outs.append([*out, sums])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
