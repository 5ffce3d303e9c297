"""The operators of the gated feed-forward block as a language model uses them, on one GPU.

Training: the norm in front of the block, the gated linear layer, the down-projection in FP8 (per tensor, delayed
scaling), then the norm behind the block with its gate, the residual sum and the next norm in one pass; and the
backward pass of all of it, the down-projection's in bfloat16.
Serving: a batch of requests with an adapter each beside the block's projections: the shared ones on bfloat16 and INT8
weights, the adapters' products added in place.

    python examples/gated_block.py

prints how far each step is from the same step in float32 torch operations.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import scaled_quantization_amd as sq  # noqa: E402

DEV, EPS = "cuda", 1e-6


def rel(a, b):
    a, b = a.detach().float(), b.detach().float()
    return float((a - b).norm() / b.norm())


def rms(v, weight):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * weight


def training(tokens=1024, width=768, hidden=2048):
    """One step of the block; returns the errors of its outputs and gradients."""
    g = torch.Generator(device=DEV).manual_seed(1)
    bf = lambda *s, std=1.0, mean=0.0: (torch.randn(s, generator=g, device=DEV) * std + mean).bfloat16()
    empty = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device=DEV)
    residual, dy, dz_next = bf(tokens, width, std=2.0), bf(tokens, width), bf(tokens, width)
    first, post, gate, pre = (bf(width, std=0.1, mean=m) for m in (1.0, 1.0, 0.5, 1.0))
    w_gate, w_up, w_down = bf(hidden, width, std=width ** -0.5), bf(hidden, width, std=width ** -0.5), \
        bf(width, hidden, std=hidden ** -0.5)

    # forward; kept for the backward pass: x, gate_pre, up_pre, h, out, z and the statistics
    x, rstd0 = empty(tokens, width), empty(tokens, t=torch.float32)
    sq.block_norm(None, residual, None, None, first, EPS, None, x, None, rstd0)
    h, gate_pre, up_pre = (empty(tokens, hidden) for _ in range(3))
    workspace = empty(max(sq.gated_linear_workspace(tokens, hidden, width),
                          sq.gated_linear_backward_workspace(tokens, hidden, width)), t=torch.uint8)
    sq.gated_linear(x, w_gate, w_up, sq.GATE_SILU, h, gate_pre, up_pre, workspace)
    state = sq.TensorState(sq.E4M3, hist_len=16, margin=1.25, initial_amax=float(h.abs().max()))
    h8, w8, w_scale = empty(tokens, hidden, t=torch.uint8), empty(width, hidden, t=torch.uint8), empty(2, t=torch.float32)
    sq.quantize_weight(w_down, sq.E4M3, sq.PER_TENSOR, w8, w_scale)
    sq.quantize_fused(h, sq.ACT_IDENTITY, sq.E4M3, sq.PER_TENSOR, state, None, h8)
    out = empty(tokens, width)
    sq.fp8_gemm_scaled(h8, sq.E4M3, w8, sq.E4M3, sq.PER_TENSOR, state.field_ptr("scale_inv"), w_scale, out)
    sq.amax_history_update(state)
    z, y = empty(tokens, width), empty(tokens, width)
    rstd1, rstd2 = empty(tokens, t=torch.float32), empty(tokens, t=torch.float32)
    sq.block_norm(out, residual, post, gate, pre, EPS, z, y, rstd1, rstd2)

    # backward: dy reaches the next norm, dz_next the residual stream past it
    dres, dout, dx, d_in = (empty(tokens, width) for _ in range(4))
    dgate, dpost, dpre, dfirst = (empty(width, t=torch.float32) for _ in range(4))
    sums = empty(2 * min(tokens, sq.NORM_PARTS) * width, t=torch.float32)
    sq.block_norm_backward(dy, dz_next, out, z, post, gate, pre, rstd1, rstd2, dres, dout, dgate, dpost, dpre, sums)
    dh, dw_down = dout @ w_down, dout.t().contiguous() @ h
    dw_gate, dw_up = empty(hidden, width), empty(hidden, width)
    sq.gated_linear_backward(dh, gate_pre, up_pre, x, w_gate, w_up, sq.GATE_SILU, workspace, dx, dw_gate, dw_up)
    sq.block_norm_backward(dx, dres, None, residual, None, None, first, None, rstd0, d_in, dpre_weight=dfirst,
                           workspace=sums)

    # the same in float32; the codes' error of the down-projection is carried over as a constant
    r, w0, wg, wu, wd, p, gt, q = (t.float().requires_grad_() for t in (residual, first, w_gate, w_up, w_down, post,
                                                                        gate, pre))
    xr = rms(r, w0)
    hr = torch.nn.functional.silu(xr @ wg.t()) * (xr @ wu.t())
    outr = hr @ wd.t()
    zr = r + gt * rms(outr + (out.float() - outr).detach(), p)
    yr = rms(zr, q)
    ((yr * dy.float()).sum() + (zr * dz_next.float()).sum()).backward()
    return {"x": rel(x, xr), "h": rel(h, hr), "FP8 down-projection": rel(out, outr), "z": rel(z, zr), "y": rel(y, yr),
            "d input": rel(d_in, r.grad), "d first norm": rel(dfirst, w0.grad), "d w_gate": rel(dw_gate, wg.grad),
            "d w_up": rel(dw_up, wu.grad), "d w_down": rel(dw_down, wd.grad), "d post norm": rel(dpost, p.grad),
            "d gate": rel(dgate, gt.grad), "d pre norm": rel(dpre, q.grad)}


def serving(tokens=40, width=768, hidden=2048, adapters=12, rank=16):
    """A decoding batch, every request with an adapter or none, through the block; returns the errors."""
    g = torch.Generator(device=DEV).manual_seed(2)
    bf = lambda *s, std=1.0: (torch.randn(s, generator=g, device=DEV) * std).bfloat16()
    x = bf(tokens, width)
    w_gate, w_up, w_down = bf(hidden, width, std=width ** -0.5), bf(hidden, width, std=width ** -0.5), \
        bf(width, hidden, std=hidden ** -0.5)
    down_a, down_b = bf(adapters, rank, hidden, std=hidden ** -0.5), bf(adapters, width, rank, std=0.2)
    scale = 0.5 + torch.rand(adapters, generator=g, device=DEV)
    index = torch.randint(-1, adapters, (tokens,), generator=g, device=DEV, dtype=torch.int32)

    # once per step: the tokens grouped by adapter, for every layer and projection
    plan = torch.empty(sq.lora_plan_size(tokens, adapters), dtype=torch.int32, device=DEV)
    sq.lora_plan(index, adapters, plan)
    h = torch.empty((tokens, hidden), dtype=x.dtype, device=DEV)
    workspace = torch.empty(max(sq.gated_linear_workspace(tokens, hidden, width),
                                sq.int8_linear_workspace(tokens, hidden) + (16 << 20),
                                sq.lora_add_workspace(tokens, width, hidden, rank, adapters)),
                            dtype=torch.uint8, device=DEV)
    sq.gated_linear(x, w_gate, w_up, sq.GATE_SILU, h, workspace=workspace)
    w8, w_scale = torch.empty_like(w_down, dtype=torch.int8), torch.empty(width, device=DEV)
    sq.quantize_int8(w_down, w8, w_scale)
    out = torch.empty_like(x)
    sq.int8_linear(h, w8, w_scale, out, workspace)
    shared = out.clone()
    sq.lora_add(h, down_a, down_b, scale, plan, out, out, workspace)          # added in place

    xf = x.float()
    hr = torch.nn.functional.silu(xf @ w_gate.float().t()) * (xf @ w_up.float().t())
    delta = torch.zeros_like(xf)
    for t, i in enumerate(index.tolist()):
        if i >= 0:
            delta[t] = scale[i] * (down_b[i].float() @ (down_a[i].float() @ hr[t]))
    return {"h": rel(h, hr), "INT8 down-projection": rel(shared, hr @ w_down.float().t()),
            "with adapters": rel(out, shared.float() + delta)}


def main():
    for title, errors in (("training, bfloat16 and FP8 against float32", training()),
                          ("serving, bfloat16 and INT8 against float32", serving())):
        print(title + ": " + ", ".join(f"{k} {v:.2e}" for k, v in errors.items()))


if __name__ == "__main__":
    main()
