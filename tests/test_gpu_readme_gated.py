"""The README's code for the gated feed-forward block, run as it stands, against the formulas in float32 torch
operations."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def rel(a, b):
    return float((a.float() - b).norm() / b.norm())


def test_gated_block_code():
    blocks = re.findall(r"```python3\n(.*?)```", open(README).read(), re.S)
    assert len(blocks) == 1
    gen = torch.Generator(device="cuda").manual_seed(3)
    bf = lambda *s, std=1.0: (torch.randn(s, generator=gen, device="cuda") * std).bfloat16()
    env = {"x": bf(1024, 768), "residual": bf(1024, 768), "dy": bf(1024, 768), "dz_next": bf(1024, 768),
           "w_gate": bf(2048, 768, std=768 ** -0.5), "w_up": bf(2048, 768, std=768 ** -0.5),
           "w_down": bf(768, 2048, std=2048 ** -0.5), "post": bf(768), "gate": bf(768), "pre": bf(768),
           "dh": bf(1024, 2048), "lora_a": bf(12, 16, 2048, std=2048 ** -0.5), "lora_b": bf(12, 768, 16, std=0.2),
           "lora_scale": torch.rand(12, generator=gen, device="cuda"),
           "index": torch.randint(-1, 12, (1024,), generator=gen, device="cuda", dtype=torch.int32)}
    exec(blocks[0], env)
    torch.cuda.synchronize()
    e = {k: v.float() for k, v in env.items() if isinstance(v, torch.Tensor)}

    # Every output is its formula of stored 16-bit inputs, rounded once to bfloat16 (off by 2^-8 of a value at
    # most); dx and the weights' gradients have each factor rounded as well.  The bound below counts three such
    # steps and the FP32 sums of both sides.
    tol = 3 * 2.0 ** -8 + 2.0 ** -12
    wg, wu, x = (e[k].clone().requires_grad_() for k in ("w_gate", "w_up", "x"))
    h = torch.nn.functional.silu(x @ wg.t()) * (x @ wu.t())
    assert rel(env["h"], h.detach()) < tol
    h.backward(e["dh"])
    for name, leaf in (("dx", x), ("dw_gate", wg), ("dw_up", wu)):
        assert rel(env[name], leaf.grad) < tol, name

    out = e["h"] @ e["w_down"].t()
    for i in range(12):
        at = (env["index"] == i).nonzero()[:, 0]
        out[at] += e["lora_scale"][i] * (e["h"][at] @ e["lora_a"][i].t() @ e["lora_b"][i].t())
    assert rel(env["out"], out) < tol

    def norm(v, weight):
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * weight
    o, r, post, gate, pre = (e[k].clone().requires_grad_() for k in ("out", "residual", "post", "gate", "pre"))
    z = r + gate * norm(o, post)
    y = norm(z, pre)
    assert rel(env["z"], z.detach()) < tol and rel(env["y"], y.detach()) < tol
    ((y * e["dy"]).sum() + (z * e["dz_next"]).sum()).backward()
    for name, leaf in (("dout", o), ("dresidual", r), ("dpost", post), ("dgate", gate), ("dpre", pre)):
        assert rel(env[name], leaf.grad) < tol, name
