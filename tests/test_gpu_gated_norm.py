"""The norms before and after a block with its gate and residual scale, and their backward pass, on the
GPU, against their 64-bit definitions (oracle/gated.py).

Tolerances, from the arithmetic: an output's last rounding is off by at most half a step of its type.  Before
it every value is binary32, U = 2^-24 per operation.  A row's sum adds at most 8 * 16 values in sequence in a thread (long
rows keep what they round off), 6 steps over a wave and 16 over its waves: S = 160 U of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

import oracle.gated as OG
import scaled_quantization_amd as sq
from gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
S = 160 * U
TYPES = [torch.bfloat16, torch.float16, torch.float32]
IDS = ["bf16", "f16", "f32"]
# one vector, odd, and both sides of every change of threads or registers per row
COLS = [1, 7, 8, 9, 100, 511, 512, 513, 1001, 1024, 1025, 1530, 1537, 2048, 2049, 4096, 4099, 8192, 8193,
        16384, 16385, 40001]
EPS, A, B = 1e-5, 1.25, -0.75


def half(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}[t]


def draw(shape, t, seed, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(t)


def f64(x):
    return x.cpu().double().numpy()


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def close(got, ref, tol, what):
    got = f64(got)
    tol = np.broadcast_to(tol, ref.shape)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {ref[bad][0]}, allowed {tol[bad][0]}")


def values(v, like):
    return np.ones(like.shape[-1]) if v is None else f64(v)


def gate_of(kind, rows, cols, t, seed=5):
    if kind == "none":
        return None
    if kind == "channel32":
        return draw(cols, torch.float32, seed, 0.2, 0.5)
    return draw((cols,) if kind == "channel" else (rows, cols), t, seed, 0.2, 0.5)


def check_forward(x, residual, post, gate, pre, z, y, r1, r2, t, what):
    fx, fr, w, g, p = f64(x), f64(residual), values(post, x), values(gate, x), values(pre, x)
    rz, _, rr1, _ = OG.block_norm(fx, fr, w, g, p, EPS, A, B)
    close(r1, rr1, (S + 4 * U) * rr1, what + " post_rstd")
    # the second norm is held to its definition on z as stored
    branch = np.abs(rz - A * fr)
    off = branch * (S + 10 * U) + 2 * U * (np.abs(A * fr) + np.abs(rz))
    close(z, rz, off + half(t) * (np.abs(rz) + off) + tiny(t), what + " z")
    if y is None:
        return
    fz = f64(z)
    rr2 = OG.rms_inverse(fz, EPS)
    close(r2, rr2, (S + 4 * U) * rr2, what + " pre_rstd")
    ref = fz * rr2[:, None] * p
    off = np.abs(ref) * (S + 8 * U)
    close(y, ref, off + half(t) * (np.abs(ref) + off) + tiny(t), what + " y")


def forward(rows, cols, t, kind, wt=None, second=True):
    wt = wt or t
    x, residual = draw((rows, cols), t, cols, 1.5, 0.25), draw((rows, cols), t, cols + 1, 2.0)
    post, pre, gate = draw(cols, wt, 1, 0.3, 1.0), draw(cols, wt, 2, 0.3, 1.0), gate_of(kind, rows, cols, t)
    z, y = (torch.full((rows, cols), float("nan"), dtype=t, device=DEV) for _ in range(2))
    r1, r2 = (torch.empty(rows, device=DEV) for _ in range(2))
    dx, dr, dpo, dg, dpr = dev(x, residual, post, gate, pre)
    sq.block_norm(dx, dr, dpo, dg, dpr, EPS, z, y if second else None, r1, r2 if second else None, A, B)
    check_forward(x, residual, post, gate, pre, z, y if second else None, r1, r2, t, f"{rows}x{cols} {kind}")


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_forward(t, cols):
    rows = 5 if cols < 5000 else 3
    forward(rows, cols, t, "channel", torch.float32 if cols % 2 else t)
    forward(rows, cols, t, "token")


@pytest.mark.parametrize("cols", [33, 768, 20000])
def test_forward_other_forms(cols):
    t = torch.bfloat16
    forward(6, cols, t, "none")
    forward(6, cols, t, "channel32")
    forward(6, cols, t, "channel", second=False)
    forward(1, cols, t, "token")
    # the norm alone, three dimensions, no statistics, no weight
    x = draw((2, 3, cols), t, 9, 2.0)
    y = torch.empty_like(x, device=DEV)
    sq.block_norm(None, x.to(DEV), None, None, None, EPS, None, y)
    v = f64(x).reshape(6, cols)
    ref = v * OG.rms_inverse(v, EPS)[:, None]
    off = np.abs(ref) * (S + 8 * U)
    close(y.reshape(6, cols), ref, off + half(t) * (np.abs(ref) + off) + tiny(t), "norm alone")
    # no weights, no gate
    r, z = draw((2, 3, cols), t, 10), torch.empty_like(x, device=DEV)
    r1, r2 = torch.empty(6, device=DEV), torch.empty(6, device=DEV)
    sq.block_norm(x.to(DEV), r.to(DEV), None, None, None, EPS, z, y, r1, r2, A, B)
    check_forward(x.reshape(6, cols), r.reshape(6, cols), None, None, None, z.reshape(6, cols),
                  y.reshape(6, cols), r1, r2, t, "no parameters")


def test_forward_many_rows():
    # more rows than one pass of the grid takes
    forward(70001, 33, torch.bfloat16, "channel")
    forward(9000, 1100, torch.float16, "token")


@pytest.mark.parametrize("cols", [100, 2056, 4099, 20000])
@pytest.mark.parametrize("kind", ["channel", "token"])
def test_forward_in_place(cols, kind):
    # z over x, the residual, or the gate per token
    rows, t = 9, torch.bfloat16
    x, residual, gate = draw((rows, cols), t, 1), draw((rows, cols), t, 2), gate_of(kind, rows, cols, t)
    post, pre = draw(cols, t, 3, 0.3, 1.0), draw(cols, t, 4, 0.3, 1.0)
    want = [torch.empty((rows, cols), dtype=t, device=DEV) for _ in range(2)]
    dx, dr, dpo, dg, dpr = dev(x, residual, post, gate, pre)
    sq.block_norm(dx, dr, dpo, dg, dpr, EPS, *want, None, None, A, B)
    for over in ("x", "residual", "gate"):
        if over == "gate" and kind != "token":
            continue
        dx, dr, dpo, dg, dpr = dev(x, residual, post, gate, pre)
        z, y = {"x": dx, "residual": dr, "gate": dg}[over], torch.empty_like(want[1])
        sq.block_norm(dx, dr, dpo, dg, dpr, EPS, z, y, None, None, A, B)
        assert torch.equal(z, want[0]) and torch.equal(y, want[1]), over


@pytest.mark.parametrize("cols", [100, 4096, 20000])
def test_forward_rows_that_are_not_finite_or_zero(cols):
    t = torch.bfloat16
    x, residual = draw((6, cols), t, 4), draw((6, cols), t, 5)
    x[1, 3], x[2, 50], x[3], residual[4] = float("nan"), float("inf"), 0.0, 0.0
    x[4] = 0.0
    z, y = (torch.empty((6, cols), dtype=t, device=DEV) for _ in range(2))
    sq.block_norm(x.to(DEV), residual.to(DEV), None, None, None, EPS, z, y)
    assert torch.isnan(z[1]).all() and torch.isnan(z[2, 50]) and torch.isnan(y[1:3]).all()
    assert torch.equal(z[3].cpu(), residual[3]) and (z[4] == 0).all() and (y[4] == 0).all()
    # a row of zeros with eps 0 is 0 times infinity
    sq.block_norm(x.to(DEV), residual.to(DEV), None, None, None, 0.0, z, y)
    assert torch.isnan(z[3]).all()
    assert torch.isfinite(y[[0, 5]]).all()


# ------------------------------------------------------------------ backward
def backward_tolerances(dy, add, x, z, w, g, p, r1, r2, t):
    """Of dz, dx, dgate per token, dpost, dpre before their last rounding (magnitudes in the place of values,
    as many U as there are operations, S for a row's mean; sums over rows come on top)."""
    dz = np.abs(add)
    off = 4 * U * dz
    dpre = 0
    if dy is not None:
        zh, c = np.abs(z * r2[:, None]), np.abs(dy * p)
        m = (c * zh).mean(1, keepdims=True)
        dz = dz + r2[:, None] * (c + zh * m)
        off = 8 * U * dz + r2[:, None] * zh * m * (S + 8 * U)
        dpre = np.abs(dy) * zh
    if x is None:
        return off, None, None, None, dpre
    xh = np.abs(x * r1[:, None])
    gw = np.abs(B * g * w)
    e, eo = dz * gw, off * gw + 6 * U * dz * gw
    m, mo = (e * xh).mean(1, keepdims=True), (eo * xh).mean(1, keepdims=True)
    m_off = mo + m * (S + 4 * U)
    dx = r1[:, None] * (eo + 4 * U * e + xh * (m_off + 6 * U * m))
    post = np.abs(B * g) * xh
    gate = np.abs(B * w) * xh
    return off, dx, gate * (off + 8 * U * dz), (post, dz, off), dpre


def check_backward(dy, add, x, z, post, gate, pre, r1, r2, out, t, kind, what):
    rows, cols = z.shape
    fd = None if dy is None else f64(dy)
    fa = np.zeros((rows, cols)) if add is None else f64(add)
    fx, fz = None if x is None else f64(x), f64(z)
    w, g, p = values(post, z), values(gate, z), values(pre, z)
    f1, f2 = None if r1 is None else f64(r1), None if r2 is None else f64(r2)
    rdr, rdx, rdg, rpo, rpr = OG.block_norm_backward(fd, fa, fx, fz, w, g, p, f1, f2, A, B)
    off, dxo, dgo, po, pr = backward_tolerances(fd, fa, fx, fz, w, g, p, f1, f2, t)
    a = 1.0 if x is None else A
    close(out["dresidual"], rdr, a * off + half(t) * (np.abs(rdr) + a * off) + 2 * U * np.abs(rdr) + tiny(t),
          what + " dresidual")
    # sums over rows: a row's share is off by its own error; adding up, a workgroup sums up to 64 rows in
    # registers, as many such sums, 4 waves, and up to 1024 partial sums in 32 and 32 steps
    rows_off = (2 * min(rows, 64) + 80) * U
    if dy is not None and out.get("dpre") is not None:
        close(out["dpre"], rpr, pr.sum(0) * (rows_off + 4 * U), what + " dpre")
    if x is None:
        return
    if out.get("dx") is not None:
        close(out["dx"], rdx, dxo + half(t) * (np.abs(rdx) + dxo) + tiny(t), what + " dx")
    wide, dz, off = po
    if out.get("dpost") is not None:
        share = wide * (off + 8 * U * dz) + rows_off * wide * dz
        close(out["dpost"], rpo, share.sum(0) + 8 * U * np.abs(rpo), what + " dpost")
    if out.get("dgate") is not None:
        if kind == "token":
            close(out["dgate"], rdg, dgo + half(t) * (np.abs(rdg) + dgo) + tiny(t), what + " dgate")
        else:
            xh = np.abs(fx * f1[:, None])
            share = np.abs(B * w) * xh * (off + 8 * U * dz + rows_off * dz)
            close(out["dgate"], rdg.sum(0), share.sum(0) + 8 * U * np.abs(rdg.sum(0)), what + " dgate")


def backward_inputs(rows, cols, t, kind, wt=None, seed=0):
    wt = wt or t
    x, z = draw((rows, cols), t, seed + 1, 1.5, 0.25), draw((rows, cols), t, seed + 2, 2.0)
    dy, add = draw((rows, cols), t, seed + 3), draw((rows, cols), t, seed + 4)
    post, pre, gate = draw(cols, wt, 6, 0.3, 1.0), draw(cols, wt, 7, 0.3, 1.0), gate_of(kind, rows, cols, t)
    r1, r2 = (torch.from_numpy(OG.rms_inverse(f64(v), EPS)).float() for v in (x, z))
    return dy, add, x, z, post, gate, pre, r1, r2


def backward(rows, cols, t, kind, wt=None, drop=(), seed=0):
    """drop: inputs and outputs that are left out."""
    names = ("dy", "add", "x", "z", "post", "gate", "pre", "r1", "r2")
    ins = dict(zip(names, backward_inputs(rows, cols, t, kind, wt, seed)))
    for n in drop:
        ins[n] = None
    out = {"dresidual": torch.full((rows, cols), float("nan"), dtype=t, device=DEV)}
    if ins["x"] is not None:
        out["dx"] = torch.full_like(out["dresidual"], float("nan"))
        out["dpost"] = torch.full((cols,), float("nan"), device=DEV)
        if kind == "token":
            out["dgate"] = torch.full_like(out["dx"], float("nan"))
        elif kind != "none":
            out["dgate"] = torch.full((cols,), float("nan"), device=DEV)
    if ins["dy"] is not None:
        out["dpre"] = torch.full((cols,), float("nan"), device=DEV)
    for n in drop:
        out.pop(n, None)
    ws = torch.full((2 * min(rows, sq.NORM_PARTS) * cols,), float("nan"), device=DEV)
    z = ins["z"]
    d = dev(*(ins[n] for n in names))
    if ins["dy"] is None:
        d[3] = d[6] = d[8] = None
    sq.block_norm_backward(*d, out["dresidual"], out.get("dx"), out.get("dgate"), out.get("dpost"),
                           out.get("dpre"), ws, A, B)
    check_backward(ins["dy"], ins["add"], ins["x"], z, ins["post"], ins["gate"], ins["pre"], ins["r1"], ins["r2"],
                   out, t, kind, f"{rows}x{cols} {kind} without {drop}")


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_backward(t, cols):
    rows = 11 if cols < 5000 else 3
    backward(rows, cols, t, "channel", torch.float32 if cols % 2 else t)
    backward(rows, cols, t, "token")


@pytest.mark.parametrize("cols", [33, 776, 2500, 9000])
def test_backward_other_forms(cols):
    t = torch.bfloat16
    backward(6, cols, t, "none")
    backward(6, cols, t, "channel32")
    backward(1, cols, t, "channel")
    backward(6, cols, t, "channel", drop=("add",))
    backward(6, cols, t, "channel", drop=("dy",))
    backward(6, cols, t, "token", drop=("dy",))
    backward(6, cols, t, "none", drop=("x", "post", "r1"))
    backward(6, cols, t, "none", drop=("x", "post", "r1", "add"))
    backward(6, cols, t, "channel", drop=("dx", "dgate"))
    backward(6, cols, t, "token", drop=("dpost", "dpre"))


@pytest.mark.parametrize("rows, cols", [(70001, 24), (5000, 520), (3000, 1100), (1500, 4104), (1300, 8200)])
def test_backward_many_rows(rows, cols):
    # each workgroup walks several rows; sums of earlier rows join; partial sums of all workgroups
    backward(rows, cols, torch.bfloat16, "channel" if cols % 100 else "token")


@pytest.mark.parametrize("cols", [100, 2060, 4099, 9001])
@pytest.mark.parametrize("kind", ["channel", "token"])
def test_backward_in_place(cols, kind):
    rows, t = 9, torch.bfloat16
    ins = backward_inputs(rows, cols, t, kind)
    ws = torch.empty(2 * rows * cols, device=DEV)

    def call(where, without_dy=False):
        d = dev(*ins)
        if without_dy:
            d[0] = d[3] = d[6] = d[8] = None
        buffers = {"dy": d[0], "add": d[1], None: None}
        out = [buffers[w] if w else torch.empty((rows, cols), dtype=t, device=DEV) for w in where]
        dgate = out[2] if kind == "token" else torch.empty(cols, device=DEV)
        sums = [torch.empty(cols, device=DEV), None if without_dy else torch.empty(cols, device=DEV)]
        sq.block_norm_backward(*d, out[0], out[1], dgate, *sums, ws, A, B)
        return [o.clone() for o in out[:2] + [dgate] + [v for v in sums if v is not None]]

    want = call((None, None, None))
    for where in (("dy", "add", None), ("add", "dy", None), ("add", None, "dy"), (None, "dy", "add")):
        if where[2] and kind != "token":
            continue
        assert all(torch.equal(a, b) for a, b in zip(call(where), want)), where
    want = call((None, None, None), True)
    for where in (("add", None, None), (None, "add", None)):
        assert all(torch.equal(a, b) for a, b in zip(call(where, True), want)), where


def test_backward_rows_that_are_not_finite_touch_no_other():
    for cols in (100, 4099, 9001):
        ins = list(backward_inputs(5, cols, torch.bfloat16, "token"))
        ins[0][1, 3], ins[2][3, 7] = float("nan"), float("inf")
        outs = [torch.empty((5, cols), dtype=torch.bfloat16, device=DEV) for _ in range(3)]
        sq.block_norm_backward(*dev(*ins), *outs)
        for o in outs:
            assert torch.isfinite(o[[0, 2, 4]]).all()
        assert torch.isnan(outs[0][1]).any()


def test_same_call_same_bits_and_replays():
    rows, cols, t = 3000, 776, torch.bfloat16
    d = dev(*backward_inputs(rows, cols, t, "channel"))
    ws = torch.empty(2 * sq.NORM_PARTS * cols, device=DEV)
    z, y = torch.empty_like(d[2]), torch.empty_like(d[2])
    r1, r2 = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    residual = draw((rows, cols), t, 50).to(DEV)
    outs = [torch.empty_like(d[2]), torch.empty_like(d[2])] + [torch.empty(cols, device=DEV) for _ in range(3)]

    def step():
        sq.block_norm(d[2], residual, d[4], d[5], d[6], EPS, z, y, r1, r2, A, B)
        sq.block_norm_backward(d[0], d[1], d[2], z, d[4], d[5], d[6], r1, r2, *outs, ws, A, B)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        d[2].copy_(draw((rows, cols), t, 60 + seed))
        ws.fill_(float("nan"))
        graph.replay()
        got = [v.clone() for v in (z, y, r1, r2, *outs)]
        torch.cuda.synchronize()
        ws.fill_(0)
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (z, y, r1, r2, *outs)))
