"""The operators around the MLP as a transformer block uses them, on one GPU.

Training: the tail of the MLP (dropout of the down-projection's output, residual sum, the
next layer norm) forward and backward, with the mask regenerated from the seed and offset.
Serving: residual sum, norm and INT8 cast in one pass, the INT8 up-projection on its codes, the
squared ReLU, and the INT8 down-projection, for a prompt and then token by token.

    python examples/mlp_block.py

prints how far each step is from the same step in float32 torch operations.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import scaled_quantization_amd as sq  # noqa: E402

DEV, EPS = "cuda", 1e-5


def rel(a, b):
    a, b = a.detach().float(), b.detach().float()
    return float((a - b).norm() / b.norm())


def training(tokens=2048, width=768, p=0.1, seed=1234, step=7, layer=3, layers=12):
    """One step of the MLP's tail; returns the errors of z, y and the gradients."""
    g = torch.Generator(device=DEV).manual_seed(1)
    bf = lambda *s, std=1.0: (torch.randn(s, generator=g, device=DEV) * std).bfloat16()
    mlp, residual, dy, dz_next = bf(tokens, width), bf(tokens, width, std=2.0), bf(tokens, width), bf(tokens, width)
    weight, bias = 1.0 + bf(width, std=0.1), bf(width, std=0.1)

    # seed and offset: the same two words give the same mask, so every layer of every step has its own
    rng = torch.tensor([seed, step * layers + layer], dtype=torch.int64, device=DEV)
    z, y, dz, dmlp = (torch.empty_like(mlp) for _ in range(4))
    mean, rstd = (torch.empty(tokens, device=DEV) for _ in range(2))
    sq.dropout_add_layer_norm(mlp, residual, p, rng, weight, bias, EPS, z, y, mean, rstd)

    # backward: dy reaches the norm, dz_next the residual stream past it
    dweight, dbias = torch.empty(width, device=DEV), torch.empty(width, device=DEV)
    workspace = torch.empty(2 * min(tokens, sq.NORM_PARTS) * width, device=DEV)
    sq.layer_norm_backward(dy, z, weight, mean, rstd, dz, dweight, dbias, workspace, dz_next, p, rng, dmlp)

    # the same in torch, with the kernel's mask read off a tensor of ones
    keep = torch.empty(tokens, width, device=DEV)
    sq.dropout_add(torch.ones_like(keep), None, p, rng, keep)
    m, r, w, b = (t.float().requires_grad_() for t in (mlp, residual, weight, bias))
    zr = r + m * keep
    yr = torch.nn.functional.layer_norm(zr, (width,), w, b, EPS)
    ((yr * dy.float()).sum() + (zr * dz_next.float()).sum()).backward()
    return {"z": rel(z, zr), "y": rel(y, yr), "d residual": rel(dz, r.grad), "d mlp": rel(dmlp, m.grad),
            "d weight": rel(dweight, w.grad), "d bias": rel(dbias, b.grad)}


class Int8Mlp:
    """norm -> up-projection -> squared ReLU -> down-projection, weights in INT8."""

    def __init__(self, norm_weight, norm_bias, up, down, max_tokens):
        self.norm = norm_weight, norm_bias
        self.up, self.down = ((torch.empty(w.shape, dtype=torch.int8, device=DEV),
                               torch.empty(w.shape[0], device=DEV)) for w in (up, down))
        for w, (codes, scale) in ((up, self.up), (down, self.down)):
            sq.quantize_int8(w, codes, scale)                            # a scale per output channel
        hidden, width = up.shape
        self.codes = torch.empty((max_tokens, width), dtype=torch.int8, device=DEV)
        self.scale = torch.empty(max_tokens, device=DEV)
        self.workspace = torch.empty(sq.int8_linear_workspace(max_tokens, hidden) + (16 << 20),
                                     dtype=torch.uint8, device=DEV)

    def __call__(self, x, residual):
        """(the block's input sum z, the MLP's output) for x and residual [tokens, width]."""
        tokens = x.shape[0]
        z, out = torch.empty_like(x), torch.empty_like(x)
        h = torch.empty((tokens, self.up[0].shape[0]), dtype=x.dtype, device=DEV)
        codes, scale = self.codes[:tokens], self.scale[:tokens]
        sq.layer_norm_quantize_int8(x, *self.norm, EPS, codes, scale, residual, z)
        sq.int8_gemm(codes, self.up[0], scale, self.up[1], h, None, self.workspace)
        h = torch.relu(h).square_()
        sq.int8_linear(h, self.down[0], self.down[1], out, self.workspace)
        return z, out


def serving(prompt=500, steps=4, width=768, hidden=2048):
    """The INT8 block against float32 for a prompt and for single tokens; returns the errors."""
    g = torch.Generator(device=DEV).manual_seed(2)
    bf = lambda *s, std=1.0: (torch.randn(s, generator=g, device=DEV) * std).bfloat16()
    weight, bias = 1.0 + bf(width, std=0.1), bf(width, std=0.1)
    up, down = bf(hidden, width, std=width ** -0.5), bf(width, hidden, std=hidden ** -0.5)
    block = Int8Mlp(weight, bias, up, down, prompt)

    def reference(x, residual):
        z = x.float() + residual.float()
        h = torch.nn.functional.layer_norm(z, (width,), weight.float(), bias.float(), EPS) @ up.float().T
        return z, torch.relu(h).square() @ down.float().T

    errors = {}
    for name, tokens in [("prompt", prompt)] + [(f"token {i}", 1) for i in range(steps)]:
        x, residual = bf(tokens, width), bf(tokens, width, std=2.0)
        z, out = block(x, residual)
        zr, outr = reference(x, residual)
        errors[name] = max(rel(z, zr), rel(out, outr))
    return errors


def main():
    for title, errors in (("training, bfloat16 against float32", training()),
                          ("serving, INT8 against float32", serving())):
        print(title + ": " + ", ".join(f"{k} {v:.2e}" for k, v in errors.items()))


if __name__ == "__main__":
    main()
