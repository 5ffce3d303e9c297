"""The gated feed-forward block's operators without a GPU: the oracle against differences and other forms,
the C ABI's symbols and refusals, and the binding's checks of its tensors.  No call here reaches a GPU."""
import os
import re

import numpy as np
import pytest
import torch

import oracle.gated as OG
import scaled_quantization_amd as sq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8dp_gated.h")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(sq.LIB_PATH):
        pytest.skip("libfp8dp.so not built")
    return sq.lib()


# ------------------------------------------------------------------ oracle
def differences(v, f, step=1e-6):
    out = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        up, down = v.copy(), v.copy()
        up[i] += step
        down[i] -= step
        out[i] = (f(up) - f(down)) / (2 * step)
    return out


def near(a, b):
    # central differences with steps of 1e-6 in 64 bits: 1e-10 of rounding over the step, 1e-12 of the third derivative
    assert np.abs(a - b).max() < 1e-7 * (1 + np.abs(b).max())


@pytest.mark.parametrize("act", OG.ACTS)
def test_activations_against_torch_and_differences(act):
    g = np.concatenate([np.linspace(-12, 12, 97), [1e-3, -40.0, 40.0]])
    f, slope = OG.activation(g, act)
    t = torch.from_numpy(g).requires_grad_()
    F = torch.nn.functional
    ref = {"silu": F.silu, "gelu": F.gelu, "gelu_tanh": lambda v: F.gelu(v, approximate="tanh"),
           "sigmoid": torch.sigmoid, "relu": F.relu, "relu2": lambda v: F.relu(v) ** 2,
           "identity": lambda v: v * 1}[act](t)
    ref.sum().backward()
    # torch forms 1 + tanh and 1 + erf, which cancel to 1e-16 of 1
    assert np.abs(f - ref.detach().numpy()).max() < 1e-13 * (1 + np.abs(f).max())
    assert np.abs(slope - t.grad.numpy()).max() < 1e-12 * (1 + np.abs(slope).max())


def test_gated_linear_gradient_against_differences():
    rng = np.random.default_rng(1)
    x, wg, wu, dh = (rng.normal(size=s) for s in ((3, 5), (4, 5), (4, 5), (3, 4)))
    for act in ("silu", "gelu", "gelu_tanh", "sigmoid", "identity"):
        _, g, u = OG.gated_linear(x, wg, wu, act)
        dx, dg, du = OG.gated_linear_backward(dh, g, u, x, wg, wu, act)
        loss = lambda a, b, c: (OG.gated_linear(a, b, c, act)[0] * dh).sum()
        near(dx, differences(x, lambda v: loss(v, wg, wu)))
        near(dg, differences(wg, lambda v: loss(x, v, wu)))
        near(du, differences(wu, lambda v: loss(x, wg, v)))


def test_block_norm_gradient_against_differences():
    rng = np.random.default_rng(2)
    x, r, gate, dy, dz = (rng.normal(size=(3, 7)) for _ in range(5))
    post, pre = rng.normal(size=7), rng.normal(size=7)
    eps, a, b = 1e-5, 1.25, -0.75

    def loss(x, r, post, gate, pre):
        z, y, _, _ = OG.block_norm(x, r, post, gate, pre, eps, a, b)
        return (y * dy).sum() + (z * dz).sum()

    for g in (gate, gate[0]):
        z, _, r1, r2 = OG.block_norm(x, r, post, g, pre, eps, a, b)
        dr, dx, dg, dpost, dpre = OG.block_norm_backward(dy, dz, x, z, post, g, pre, r1, r2, a, b)
        near(dr, differences(r, lambda v: loss(x, v, post, g, pre)))
        near(dx, differences(x, lambda v: loss(v, r, post, g, pre)))
        near(dg if g.ndim == 2 else dg.sum(0), differences(g, lambda v: loss(x, r, post, v, pre)))
        near(dpost, differences(post, lambda v: loss(x, r, v, g, pre)))
        near(dpre, differences(pre, lambda v: loss(x, r, post, g, v)))


def test_lora_oracle():
    rng = np.random.default_rng(3)
    x, a, b, base = (rng.normal(size=s) for s in ((5, 6), (3, 2, 6), (3, 4, 2), (5, 4)))
    y, _ = OG.lora_add(x, a, b, np.array([1.0, 2.0, 3.0]), [0, -1, 2, 3, 2], base, [2, 1, 1])
    assert np.array_equal(y[[1, 3]], base[[1, 3]])
    near(y[0], base[0] + b[0] @ a[0] @ x[0])
    near(y[2], base[2] + 3 * b[2][:, :1] @ a[2][:1] @ x[2])


# ------------------------------------------------------------------ C ABI
def test_library_exports_every_declared_symbol(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^(?:int|int64_t)\s+(\w+)\s*\(", text, flags=re.M))
    assert names == {"gated_linear_workspace", "gated_linear", "gated_linear_backward_workspace",
                     "gated_linear_backward", "block_norm", "block_norm_backward", "lora_plan_size",
                     "lora_plan", "lora_add_workspace", "lora_add"}
    assert all(hasattr(L, n) and n in sq._SIGS for n in names)
    gates = re.findall(r"FP8DP_GATE_(\w+) = (\d+)", text)
    assert len(gates) == 7 and all(getattr(sq, "GATE_" + n) == int(v) for n, v in gates)
    assert tuple(n.lower() for n, _ in gates) == OG.ACTS


def test_c_refusals(L):
    def refused(rc, word):
        assert rc == -1 and word in L.fp8dp_last_error(), (rc, L.fp8dp_last_error())

    nan, inf = float("nan"), float("inf")
    # gated_linear(x, wg, wu, M, N, K, dt, act, h, gate, up, ws, bytes, stream)
    gl = lambda x=16, wg=16, M=4, N=8, K=8, dt=0, act=0, h=32, g=None, u=None, ws=None, room=0: \
        L.gated_linear(x, wg, 16, M, N, K, dt, act, h, g, u, ws, room, None)
    for kw in ({"x": None}, {"wg": None}, {"h": None}):
        refused(gl(**kw), b"non-NULL")
    for kw in ({"M": 0}, {"N": 0}, {"K": 0}, {"M": -1}, {"M": (1 << 24) + 1}, {"N": (1 << 20) + 1},
               {"K": (1 << 20) + 1}):
        refused(gl(**kw), b"must be")
    for dt in (2, 3, -1):
        refused(gl(dt=dt), b"type")
    for act in (7, -1):
        refused(gl(act=act), b"activation")
    refused(gl(g=48), b"together")
    refused(gl(u=48), b"together")
    refused(gl(g=32, u=48), b"different")
    refused(gl(g=48, u=48), b"different")
    refused(gl(h=16), b"different")
    refused(gl(g=16, u=48), b"different")
    refused(gl(x=17), b"aligned")
    refused(gl(g=49, u=64), b"aligned")
    refused(gl(ws=24, room=64), b"workspace")
    refused(gl(ws=16, room=-1), b"workspace")
    # gated_linear_backward(dh, gate, up, x, wg, wu, M, N, K, dt, act, dx, dwg, dwu, ws, bytes, stream)
    need = L.gated_linear_backward_workspace(4, 8, 8)
    assert need >= 4 * 2 * 8 * 2
    gb = lambda dh=16, up=16, M=4, dt=0, act=0, dx=32, dwg=48, dwu=64, ws=16, room=need: \
        L.gated_linear_backward(dh, 16, up, 16, 16, 16, M, 8, 8, dt, act, dx, dwg, dwu, ws, room, None)
    for kw in ({"dh": None}, {"up": None}, {"ws": None}):
        refused(gb(**kw), b"non-NULL")
    refused(gb(M=0), b"must be")
    refused(gb(dt=2), b"type")
    refused(gb(act=9), b"activation")
    refused(gb(dwg=None), b"together")
    refused(gb(dx=None, dwg=None, dwu=None), b"computed")
    refused(gb(room=need - 1), b"%d bytes" % need)
    refused(gb(ws=8), b"workspace")
    refused(gb(dx=33), b"aligned")
    refused(gb(dx=16), b"outputs")
    refused(gb(dwu=48), b"outputs")
    # block_norm(x, residual, post, gate, per_token, pre, rows, cols, dt, wt, gt, a, b, eps, z, y, r1, r2, stream)
    bn = lambda x=16, res=16, post=16, gate=16, tok=0, rows=4, cols=8, dt=0, wt=0, gt=0, a=1.0, b=1.0, \
        eps=1e-5, z=32, y=64, r1=None: L.block_norm(x, res, post, gate, tok, 16, rows, cols, dt, wt, gt, a, b,
                                                    eps, z, y, r1, None, None)
    for kw in ({"res": None}, {"x": None}, {"z": None}, {"x": None, "z": None, "y": None}):
        refused(bn(**kw), b"non-NULL")
    for kw in ({"post": 16, "gate": None}, {"post": None, "gate": 16}, {"post": None, "gate": None, "r1": 16}):
        refused(bn(x=None, z=None, **kw), b"belong")
    for r, c in ((0, 8), (4, 0), (-1, 8), (1 << 31, 8), (4, (1 << 30) + 1)):
        refused(bn(rows=r, cols=c), b"rows")
    for kw in ({"dt": 3}, {"wt": 1}, {"gt": 1}):
        refused(bn(**kw), b"type")
    refused(bn(tok=1, gt=2), b"per token")
    for kw in ({"eps": -1e-9}, {"eps": nan}, {"a": inf}, {"b": nan}):
        refused(bn(**kw), b"finite")
    for kw in ({"x": 17}, {"z": 33}, {"gate": 17}, {"gate": 18, "gt": 2}, {"r1": 18}):
        refused(bn(**kw), b"aligned")
    refused(bn(z=64), b"must not be")
    refused(bn(y=16), b"must not be")
    refused(bn(y=16, x=96, gate=16, tok=1, res=112), b"must not be")
    refused(bn(x=None, z=None, post=None, gate=None, y=16), b"must not be")
    # block_norm_backward(dy, add, x, z, post, gate, per_token, pre, r1, r2, rows, cols, dt, wt, gt, a, b, dres, dx,
    #                     dgate, dpost, dpre, ws, stream)
    bb = lambda dy=16, add=16, x=128, z=144, post=16, gate=16, tok=0, pre=16, r1=16, r2=16, rows=4, dt=0, wt=0, \
        gt=0, a=1.0, dres=32, dx=48, dgate=64, dpost=80, dpre=96, ws=112: L.block_norm_backward(
            dy, add, x, z, post, gate, tok, pre, r1, r2, rows, 8, dt, wt, gt, a, 1.0, dres, dx, dgate, dpost, dpre,
            ws, None)
    no_x = dict(x=None, post=None, gate=None, dx=None, dgate=None, dpost=None)
    refused(bb(dres=None), b"non-NULL")
    refused(bb(dy=None, add=None), b"non-NULL")
    refused(bb(dy=None, pre=None, dpre=None, **no_x), b"non-NULL")
    for kw in ({"z": None}, {"r2": None}, {"dy": None}, {"dy": None, "pre": None}):
        refused(bb(**kw), b"dy comes")
    refused(bb(r1=None), b"x comes")
    for k in no_x:
        if k != "x":
            refused(bb(**{**no_x, k: 160}), b"x comes")
    refused(bb(gate=None), b"needs the gate")
    refused(bb(rows=0), b"rows")
    refused(bb(dt=5), b"type")
    refused(bb(tok=1, gt=2), b"per token")
    refused(bb(a=nan), b"finite")
    refused(bb(ws=None), b"workspace")
    for kw in ({"dx": 49}, {"dgate": 66}, {"dpost": 82}, {"ws": 114}):
        refused(bb(**kw), b"aligned")
    for kw in ({"dx": 32}, {"dres": 128}, {"dx": 144}, {"tok": 1, "dgate": 48}, {"tok": 1, "dgate": 16}):
        refused(bb(**kw), b"different")
    # lora
    assert L.lora_plan_size(0, 4) == L.lora_plan_size(4, 0) == L.lora_plan_size((1 << 22) + 1, 4) == -1
    assert L.lora_plan_size(4, 2049) == -1 and L.lora_plan_size(40, 3) == 4 + 40 + 2 * (1 + 4)
    refused(L.lora_plan(None, 4, 4, 16, None), b"non-NULL")
    refused(L.lora_plan(16, 4, 4, None, None), b"non-NULL")
    refused(L.lora_plan(16, 0, 4, 16, None), b"tokens")
    refused(L.lora_plan(16, 4, 2049, 16, None), b"adapters")
    refused(L.lora_plan(18, 4, 4, 16, None), b"aligned")
    for args in ((0, 8, 8, 4, 2), (4, 0, 8, 4, 2), (4, 8, 0, 4, 2), (4, 8, 8, 0, 2), (4, 8, 8, 257, 2), (4, 8, 8, 4, 0)):
        assert L.lora_add_workspace(*args) == -1
    need = L.lora_add_workspace(4, 8, 8, 4, 2)
    assert need >= 4 * 16 * 4
    # lora_add(x, a, b, scale, ranks, plan, base, tokens, N, K, rank, adapters, dt, y, ws, bytes, stream)
    la = lambda x=16, s=16, ranks=None, plan=16, base=None, tokens=4, N=8, K=8, rank=4, adapters=2, dt=0, y=32, \
        ws=16, room=need: L.lora_add(x, 16, 16, s, ranks, plan, base, tokens, N, K, rank, adapters, dt, y, ws, room,
                                     None)
    for kw in ({"x": None}, {"s": None}, {"plan": None}, {"y": None}, {"ws": None}):
        refused(la(**kw), b"non-NULL")
    refused(la(tokens=0), b"tokens")
    refused(la(adapters=4096), b"adapters")
    for kw in ({"N": 0}, {"K": 0}, {"rank": 0}, {"rank": 257}, {"N": (1 << 20) + 1}):
        refused(la(**kw), b"must be")
    refused(la(dt=2), b"type")
    for kw in ({"x": 17}, {"s": 18}, {"ranks": 18}, {"plan": 18}, {"base": 17}):
        refused(la(**kw), b"aligned")
    refused(la(room=need - 1), b"%d bytes" % need)
    refused(la(ws=24), b"workspace")
    refused(la(y=16), b"must not be")


# ------------------------------------------------------------------ binding
def test_binding_refusals(L):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    f32, u8 = torch.zeros, lambda n: torch.zeros(n, dtype=torch.uint8)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    E = sq.Fp8dpError
    x, w, h = bf(4, 16), bf(8, 16), bf(4, 8)
    gl, gb, bn, bb = sq.gated_linear, sq.gated_linear_backward, sq.block_norm, sq.block_norm_backward
    la = lambda **kw: sq.lora_add(**{**dict(x=x, a=bf(2, 3, 16), b=bf(2, 8, 3), scale=f32(2), plan=i32(
        sq.lora_plan_size(4, 2)), base=h, y=h, workspace=u8(1 << 12)), **kw})
    v, r = bf(16), f32(4)
    for call, word in (
            (lambda: gl(x.int(), w, w, 0, h), "x: expected bfloat16"),
            (lambda: gl(x, bf(8, 15), w, 0, h), "weights must be"),
            (lambda: gl(x, bf(16), w, 0, h), "weights must be"),
            (lambda: gl(x, w, bf(9, 16), 0, h), "w_up: expected"),
            (lambda: gl(x, w.half(), w, 0, h), "w_gate: expected"),
            (lambda: gl(x, w, w, 0, bf(4, 9)), "h: expected"),
            (lambda: gl(x, w, w, 0, h, h.half(), h), "gate: expected"),
            (lambda: gl(x, w, w, 0, h, h, bf(8, 4)), "up: expected"),
            (lambda: gl(x, w, w, 0, h), "device tensor"),
            (lambda: gb(bf(4, 9), h, h, x, w, w, 0, u8(99)), "dh: expected"),
            (lambda: gb(h, h, h, x, w, w, 0, u8(99), bf(4, 8)), "dx: expected"),
            (lambda: gb(h, h, h, x, w, w, 0, u8(99), x, f32(8, 16), w), "dw_gate: expected"),
            (lambda: gb(h, h, h, x, w, w, 0, u8(99), x, w, bf(16, 8)), "dw_up: expected"),
            (lambda: bn(bf(4, 8), x, v, None, v, 1e-5, x, x), "x: expected"),
            (lambda: bn(x, x, v, None, f32(16), 1e-5, x, x), "all"),
            (lambda: bn(x, x, bf(8), None, v, 1e-5, x, x), "16 values"),
            (lambda: bn(x, x, v, bf(8), v, 1e-5, x, x), "gate: expected 16"),
            (lambda: bn(x, x, v, v.half(), v, 1e-5, x, x), "gate: expected"),
            (lambda: bn(x, x, v, f32(4, 16), v, 1e-5, x, x), "gate: expected"),
            (lambda: bn(x, x, v, bf(4, 1), v, 1e-5, x, x), "gate: expected"),
            (lambda: bn(x, x, v, None, v, 1e-5, x.float(), x), "z: expected"),
            (lambda: bn(x, x, v, None, v, 1e-5, x, bf(4, 17)), "y: expected"),
            (lambda: bn(x, x, v, None, v, 1e-5, x, x, f32(3)), "post_rstd: expected 4"),
            (lambda: bb(x, x, x, bf(4, 8), v, None, v, r, r, x), "z: expected"),
            (lambda: bb(x, x, x, x, v, None, v, f32(5), r, x), "post_rstd: expected 4"),
            (lambda: bb(x, x, x, x, v, v, v, r, r, x, x, v), "dgate: expected 16 float32"),
            (lambda: bb(x, x, x, x, v, x, v, r, r, x, x, f32(4, 16)), "dgate: expected"),
            (lambda: bb(x, x, x, x, v, None, v, r, r, x, dpost_weight=v), "dpost_weight: expected"),
            (lambda: bb(x, x, x, x, v, None, v, r, r, x, dpre_weight=f32(16), workspace=f32(127)), "workspace"),
            (lambda: sq.lora_plan(torch.zeros(4, dtype=torch.int64), 2, i32(99)), "index: expected"),
            (lambda: sq.lora_plan(i32(4), 2, i32(5)), "plan: expected"),
            (lambda: sq.lora_plan(i32(4), 2049, i32(5)), "out of range"),
            (lambda: sq.lora_plan_size(0, 2), "out of range"),
            (lambda: sq.lora_add_workspace(4, 8, 8, 300, 2), "out of range"),
            (lambda: la(a=bf(3, 16)), "a must be"),
            (lambda: la(a=bf(2, 3, 15)), "a: expected"),
            (lambda: la(b=bf(2, 3, 8)), "b: expected"),
            (lambda: la(b=bf(3, 8, 3)), "b: expected"),
            (lambda: la(base=bf(4, 9)), "base: expected"),
            (lambda: la(y=h.half()), "y: expected"),
            (lambda: la(scale=f32(3)), "scale: expected 2"),
            (lambda: la(ranks=f32(2)), "ranks|expected 2 int32"),
            (lambda: la(plan=i32(7)), "plan: expected"),
            (lambda: la(), "device tensor"),
    ):
        with pytest.raises(E, match=word):
            call()
