"""Cases of the gated feed-forward block's operators: the gated linear layer (both projections, the
activation and the product) and its gradients, the norms before and after a block with its gate
and residual scale and their gradients, and low-rank adapters of many requests beside a shared
projection.

`run` computes them in elementary torch operations, or, where `own` is true, through
scaled_quantization_amd's entry points.

Formulas, rows r of rows x cols inputs, rms(v) = v / sqrt(mean(v^2) + eps) over a row:
  gated       g = x Wg^T, u = x Wu^T, h = f(g) u; f(g) is g sigmoid(g) (silu), g Phi(g) with the normal
              distribution's Phi (gelu) or its tanh form (gelu_tanh), sigmoid(g), max(g, 0) (relu) or
              max(g, 0)^2 (relu2)
  gated_grad  dg = dh u f'(g), du = dh f(g), dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x
  norm        p = rms(x) w_post, z = a residual + b gate p, y = rms(z) w_pre; gate: one value per
              channel, one per token and channel, or 1
  norm_grad   with xh = x post_rstd, zh = z pre_rstd, c = dy w_pre:
              dz = dz_add + pre_rstd (c - zh mean(c zh)), dresidual = a dz, dw_pre = sum dy zh,
              dgate = b dz p (summed over the tokens where they share it), e = b gate dz,
              dw_post = sum e xh, dx = post_rstd (e w_post - xh mean(e w_post xh))
  lora        y[t] = base[t] + scale[i] B_i (A_i x[t]) with i = index[t]; y[t] = base[t] where i < 0;
              of adapter i the first ranks[i] of R rows of A and columns of B count
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
ACTS = ["silu", "gelu", "gelu_tanh", "sigmoid", "relu", "relu2"]


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of a decoding sequence in a small model: latency
        {"name": "gated_one_token", "op": "gated", "rows": 1, "n": 2048, "k": 768, "type": "bf16",
         "act": "silu", "train": False},
        # a decoding batch in a wide model: the weights' bytes
        {"name": "gated_batch", "op": "gated", "rows": 48, "n": 16384, "k": 4096, "type": "bf16",
         "act": "gelu_tanh", "train": False},
        # a prompt of ragged length and odd widths: no row but the first is aligned
        {"name": "gated_odd", "op": "gated", "rows": 777, "n": 1023, "k": 1001, "type": "f16",
         "act": "gelu", "train": False},
        # a wide model's training step: pre-activations kept for the backward pass
        {"name": "gated_large", "op": "gated", "rows": 16384, "n": 8192, "k": 4096, "type": "bf16",
         "act": "silu", "train": True},
        # 8 sequences x 2048 tokens of model width 768: the backward pass of the training benchmark's step
        {"name": "gated_grad_train", "op": "gated_grad", "rows": 16384, "n": 2048, "k": 768,
         "type": "bf16", "act": "silu"},
        # the backward pass at ragged sizes
        {"name": "gated_grad_odd", "op": "gated_grad", "rows": 1025, "n": 1023, "k": 1001, "type": "f16",
         "act": "gelu_tanh"},
        # between two blocks while one sequence decodes: latency
        {"name": "norm_one_token", "op": "norm", "rows": 1, "cols": 4096, "type": "bf16",
         "gate": "channel"},
        # the training benchmark's tokens, a learned gate per channel
        {"name": "norm_train", "op": "norm", "rows": 16384, "cols": 768, "type": "bf16",
         "gate": "channel"},
        # its backward pass at a ragged token count and an odd width, in 16 bits of the other kind
        {"name": "norm_grad_odd", "op": "norm_grad", "rows": 2049, "cols": 1001, "type": "f16",
         "gate": "channel"},
        # a wide model's backward pass, larger than every cache, with a gate per token
        {"name": "norm_grad_wide", "op": "norm_grad", "rows": 16384, "cols": 4096, "type": "bf16",
         "gate": "token"},
        # a decoding batch, every request with an adapter of its own
        {"name": "lora_decode", "op": "lora", "rows": 64, "n": 4096, "k": 4096, "rank": 16,
         "adapters": 64, "ragged": False, "packed": False, "type": "bf16"},
        # packed prompts of a few adapters with ranks of their own
        {"name": "lora_prompts", "op": "lora", "rows": 5003, "n": 4096, "k": 4096, "rank": 64,
         "adapters": 8, "ragged": True, "packed": True, "type": "bf16"},
    ]


def _size(rng, low, high):
    """A whole number, spread over its logarithm; two of three are multiples of 8."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if v >= 16 and rng.random() < 0.67:
        v -= v % 8
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_grad", "norm", "norm_grad", "lora"])
    case = {"op": op, "type": rng.choice(["bf16", "bf16", "f16"])}
    if op == "gated":
        case.update(rows=_size(rng, 1, 16384), n=_size(rng, 16, 8192), k=_size(rng, 16, 4096),
                    act=rng.choice(ACTS), train=rng.random() < 0.4)
    elif op == "gated_grad":
        case.update(rows=_size(rng, 1, 16384), n=_size(rng, 16, 4096), k=_size(rng, 16, 2048),
                    act=rng.choice(ACTS))
    elif op == "lora":
        rank = rng.choice([4, 8, 8, 16, 16, 32, 64, 128, 7, 20])
        case.update(rows=_size(rng, 1, 8192), n=_size(rng, 64, 8192), k=_size(rng, 64, 8192), rank=rank,
                    adapters=_size(rng, 1, min(256, 4096 // rank)), ragged=rng.random() < 0.5,
                    packed=rng.random() < 0.5)
    else:
        case["type"] = rng.choice(["bf16", "bf16", "f16", "f32"])
        case["cols"] = _size(rng, 64, 16384)
        case["rows"] = _size(rng, 1, min(65536, (1 << 25) // case["cols"]))
        case["gate"] = rng.choice(["none", "channel", "token"])
    return case


def work(case):
    r, e = case["rows"], BYTES[case["type"]]
    if case["op"] == "gated":
        n, k = case["n"], case["k"]
        return {"bytes": e * (r * k + 2 * n * k + r * n * (3 if case["train"] else 1)),
                "flops": 4 * r * n * k}
    if case["op"] == "gated_grad":
        n, k = case["n"], case["k"]
        return {"bytes": e * (3 * r * n + 2 * r * k + 4 * n * k), "flops": 8 * r * n * k}
    if case["op"] == "lora":
        n, k, rank = case["n"], case["k"], case["rank"]
        used = min(r, case["adapters"])
        return {"bytes": e * (r * (k + 2 * n) + used * rank * (k + n)) + 4 * (r + 2 * used),
                "flops": 2 * r * rank * (k + n)}
    c, gate = case["cols"], case["gate"]
    per_token, params = gate == "token", 3 if gate == "channel" else 2
    if case["op"] == "norm":
        return {"bytes": e * r * c * (4 + per_token) + e * params * c + 8 * r, "flops": 0}
    # dy, dz_add, x, z, dresidual, dx; gate and dgate
    return {"bytes": e * r * c * (6 + 2 * per_token) + (e + 4) * params * c + 8 * r, "flops": 0}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t, r, op = TYPES[case["type"]], case["rows"], case["op"]

    def normal(*shape, std=1.0, mean=0.0, to=t):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(to)

    def empty(*shape, to=t):
        return torch.empty(shape, dtype=to, device="cuda")

    s = {"case": dict(case)}
    if op in ("gated", "gated_grad"):
        n, k = case["n"], case["k"]
        # behind a norm, a few channels much larger than the rest
        channel = torch.where(torch.rand(k, generator=g, device="cuda") < 0.01, 6.0, 1.0)
        s["x"] = (torch.randn((r, k), generator=g, device="cuda") * channel).to(t)
        s["w_gate"], s["w_up"] = normal(n, k, std=k ** -0.5), normal(n, k, std=k ** -0.5)
        if op == "gated":
            s["h"] = empty(r, n)
            if case["train"]:
                s["gate"], s["up"] = empty(r, n), empty(r, n)
        else:
            # what the forward pass kept
            s["gate"] = (s["x"].float() @ s["w_gate"].float().t()).to(t)
            s["up"] = (s["x"].float() @ s["w_up"].float().t()).to(t)
            s["dh"] = normal(r, n, std=0.05)
            s["dx"] = empty(r, k)
            s["dw_gate"], s["dw_up"] = (empty(n, k) for _ in range(2))
        if own:
            import scaled_quantization_amd as sq
            size = sq.gated_linear_workspace if op == "gated" else sq.gated_linear_backward_workspace
            s["workspace"] = empty(size(r, n, k), to=torch.uint8)
        return s
    if op == "lora":
        n, k, rank, adapters = case["n"], case["k"], case["rank"], case["adapters"]
        s["x"], s["base"] = normal(r, k), normal(r, n)
        s["a"], s["b"] = normal(adapters, rank, k, std=k ** -0.5), normal(adapters, n, rank, std=0.1)
        s["scale"] = 0.25 + 2.0 * torch.rand(adapters, generator=g, device="cuda")
        if case["ragged"]:
            s["ranks"] = torch.randint(1, rank + 1, (adapters,), generator=g, device="cuda",
                                       dtype=torch.int32)
        order = torch.randperm(adapters, generator=g, device="cuda")
        at = torch.arange(r, device="cuda")
        if case["packed"]:
            # sequences of unequal length one after another
            cuts = torch.randint(0, r + 1, (2 * adapters - 1,), generator=g, device="cuda")
            at = (at[:, None] >= cuts[None, :]).sum(1)
        index = order[at % adapters]
        # a request in eight has no adapter
        s["index"] = torch.where(at % 8 == 7, -1, index).to(torch.int32)
        s["y"] = empty(r, n)
        if own:
            import scaled_quantization_amd as sq
            # made once per step, for all layers
            s["plan"] = empty(sq.lora_plan_size(r, adapters), to=torch.int32)
            sq.lora_plan(s["index"], adapters, s["plan"])
            s["workspace"] = empty(sq.lora_add_workspace(r, n, k, rank, adapters), to=torch.uint8)
        return s
    c = case["cols"]
    s["x"], s["residual"] = normal(r, c, std=1.5, mean=0.25), normal(r, c, std=2.0)
    s["post"], s["pre"] = normal(c, std=0.1, mean=1.0), normal(c, std=0.1, mean=1.0)
    s["gate"] = None
    if case["gate"] == "channel":
        s["gate"] = normal(c, std=0.1, mean=0.5)
    if case["gate"] == "token":
        s["gate"] = torch.sigmoid(torch.randn((r, c), generator=g, device="cuda")).to(t)
    s["residual_scale"], s["branch_scale"] = 1.25, 0.75
    s["post_rstd"], s["pre_rstd"] = empty(r, to=torch.float32), empty(r, to=torch.float32)
    if op == "norm":
        s["z"], s["y"] = empty(r, c), empty(r, c)
        return s
    # what the forward pass kept
    x = s["x"].float()
    s["post_rstd"] = torch.rsqrt(x.square().mean(1) + EPS)
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    z = s["residual"].float() * s["residual_scale"] + \
        s["branch_scale"] * gate * (x * s["post_rstd"][:, None] * s["post"].float())
    s["z"] = z.to(t)
    s["pre_rstd"] = torch.rsqrt(s["z"].float().square().mean(1) + EPS)
    del s["residual"]
    s["dy"], s["dz_add"] = normal(r, c, std=0.02), normal(r, c, std=0.02)
    s["dresidual"], s["dx"] = empty(r, c), empty(r, c)
    s["dgate"] = None
    if case["gate"] == "channel":
        s["dgate"] = empty(c, to=torch.float32)
    if case["gate"] == "token":
        s["dgate"] = empty(r, c)
    s["dpost"], s["dpre"] = empty(c, to=torch.float32), empty(c, to=torch.float32)
    # two partial sums per column and workgroup
    s["workspace"] = empty(2 * min(r, 1024) * c, to=torch.float32)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import scaled_quantization_amd as sq
    case = s["case"]
    op = case["op"]
    if op in ("gated", "gated_grad"):
        act = {"silu": sq.GATE_SILU, "gelu": sq.GATE_GELU, "gelu_tanh": sq.GATE_GELU_TANH,
               "sigmoid": sq.GATE_SIGMOID, "relu": sq.GATE_RELU, "relu2": sq.GATE_RELU2}[case["act"]]
    if op == "gated":
        sq.gated_linear(s["x"], s["w_gate"], s["w_up"], act, s["h"], s.get("gate"), s.get("up"),
                        s["workspace"])
        return (s["h"], s["gate"], s["up"]) if case["train"] else s["h"]
    if op == "gated_grad":
        sq.gated_linear_backward(s["dh"], s["gate"], s["up"], s["x"], s["w_gate"], s["w_up"], act,
                                 s["workspace"], s["dx"], s["dw_gate"], s["dw_up"])
        return s["dx"], s["dw_gate"], s["dw_up"]
    if op == "norm":
        sq.block_norm(s["x"], s["residual"], s["post"], s["gate"], s["pre"], EPS, s["z"], s["y"],
                      s["post_rstd"], s["pre_rstd"], s["residual_scale"], s["branch_scale"])
        return s["z"], s["y"], s["post_rstd"], s["pre_rstd"]
    if op == "norm_grad":
        sq.block_norm_backward(s["dy"], s["dz_add"], s["x"], s["z"], s["post"], s["gate"], s["pre"],
                               s["post_rstd"], s["pre_rstd"], s["dresidual"], s["dx"], s["dgate"],
                               s["dpost"], s["dpre"], s["workspace"], s["residual_scale"],
                               s["branch_scale"])
        grads = s["dresidual"], s["dx"], s["dpost"], s["dpre"]
        return grads if s["gate"] is None else grads + (s["dgate"],)
    sq.lora_add(s["x"], s["a"], s["b"], s["scale"], s["plan"], s["base"], s["y"], s["workspace"],
                s.get("ranks"))
    return s["y"]


def _activation(g, act):
    """f(g) and f'(g)."""
    if act in ("silu", "sigmoid"):
        p = 1.0 / (1.0 + torch.exp(-g))
        if act == "silu":
            return g * p, p * (1.0 + g * (1.0 - p))
        return p, p * (1.0 - p)
    if act == "gelu":
        p = 0.5 * (1.0 + torch.erf(g * 0.5 ** 0.5))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (0.5 / math.pi) ** 0.5
    if act == "gelu_tanh":
        c = (2.0 / math.pi) ** 0.5
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        slope = 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)
        return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + slope
    top = torch.clamp(g, min=0.0)
    return (top, (g > 0).to(g.dtype)) if act == "relu" else (top * top, 2.0 * top)


def _plain(s):
    case = s["case"]
    op, t = case["op"], s["x"].dtype
    x = s["x"].float()
    if op == "gated":
        g, u = x @ s["w_gate"].float().t(), x @ s["w_up"].float().t()
        h = (_activation(g, case["act"])[0] * u).to(t)
        return (h, g.to(t), u.to(t)) if case["train"] else h
    if op == "gated_grad":
        dh = s["dh"].float()
        f, slope = _activation(s["gate"].float(), case["act"])
        dg, du = dh * s["up"].float() * slope, dh * f
        return ((dg @ s["w_gate"].float() + du @ s["w_up"].float()).to(t), (dg.t() @ x).to(t),
                (du.t() @ x).to(t))
    if op == "lora":
        adapters, rank, k = s["a"].shape
        a, b = s["a"].float(), s["b"].float()
        if "ranks" in s:
            counts = torch.arange(rank, device=x.device)[None, :] < s["ranks"][:, None]
            a = torch.where(counts[:, :, None], a, 0.0)
            b = torch.where(counts[:, None, :], b, 0.0)
        mine = s["index"][:, None] == torch.arange(adapters, device=x.device)
        v = (x @ a.reshape(adapters * rank, k).t()).reshape(-1, adapters, rank)
        v = torch.where(mine[:, :, None], v * s["scale"][None, :, None], 0.0)
        b = b.permute(0, 2, 1).reshape(adapters * rank, -1)
        return (s["base"].float() + v.reshape(-1, adapters * rank) @ b).to(t)
    post, pre = s["post"].float(), s["pre"].float()
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    a, b = s["residual_scale"], s["branch_scale"]
    if op == "norm":
        post_rstd = 1.0 / torch.sqrt((x * x).mean(1) + EPS)
        z = (a * s["residual"].float() + b * gate * (x * post_rstd[:, None] * post)).to(t)
        zf = z.float()
        pre_rstd = 1.0 / torch.sqrt((zf * zf).mean(1) + EPS)
        return z, (zf * pre_rstd[:, None] * pre).to(t), post_rstd, pre_rstd
    post_rstd, pre_rstd = s["post_rstd"][:, None], s["pre_rstd"][:, None]
    xh, zh, dy = x * post_rstd, s["z"].float() * pre_rstd, s["dy"].float()
    c = dy * pre
    dz = s["dz_add"].float() + pre_rstd * (c - zh * (c * zh).mean(1, keepdim=True))
    e = b * gate * dz
    ew = e * post
    dx = post_rstd * (ew - xh * (ew * xh).mean(1, keepdim=True))
    grads = (a * dz).to(t), dx.to(t), (e * xh).sum(0), (dy * zh).sum(0)
    if case["gate"] == "channel":
        return grads + ((b * dz * xh * post).sum(0),)
    if case["gate"] == "token":
        return grads + ((b * dz * xh * post).to(t),)
    return grads


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definitions in 64 bits, on the GPU."""
    s = prepare(case, seed)
    op, t = case["op"], s["x"].dtype
    x = s["x"].double()
    if op in ("gated", "gated_grad"):
        wg, wu = s["w_gate"].double(), s["w_up"].double()
        g = torch.matmul(x, wg.t().contiguous()) if op == "gated" else s["gate"].double()
        act = case["act"]
        if act == "silu":
            p = torch.sigmoid(g)
            f, slope = g * p, p + g * p * (1 - p)
        elif act == "sigmoid":
            f = torch.sigmoid(g)
            slope = f * (1 - f)
        elif act == "gelu":
            phi = torch.special.ndtr(g)
            f, slope = g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        elif act == "gelu_tanh":
            # (1 + tanh(v)) / 2 = sigmoid(2 v)
            v = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
            p = torch.sigmoid(v)
            f = g * p
            slope = p + g * p * (1 - p) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * g ** 2)
        elif act == "relu":
            f, slope = torch.relu(g), torch.heaviside(g, torch.zeros_like(g))
        else:
            f, slope = torch.relu(g) ** 2, 2 * torch.relu(g)
        if op == "gated":
            u = torch.matmul(x, wu.t().contiguous())
            return (f * u, g, u) if case["train"] else f * u
        dh = s["dh"].double()
        dg, du = dh * s["up"].double() * slope, dh * f
        dx = torch.matmul(dg, wg) + torch.matmul(du, wu)
        return dx, torch.matmul(dg.t().contiguous(), x), torch.matmul(du.t().contiguous(), x)
    if op == "lora":
        y = s["base"].double()
        index = s["index"].tolist()
        ranks = s["ranks"].tolist() if "ranks" in s else [case["rank"]] * case["adapters"]
        scale = s["scale"].double()
        for i in sorted(set(index) - {-1}):
            rows = [j for j, v in enumerate(index) if v == i]
            v = torch.matmul(x[rows], s["a"][i, :ranks[i]].double().t().contiguous())
            y[rows] += torch.matmul(v, s["b"][i, :, :ranks[i]].double().t().contiguous()) * scale[i]
        return y
    post, pre = s["post"].double(), s["pre"].double()
    gate = torch.ones_like(post) if s["gate"] is None else s["gate"].double()
    a, b = s["residual_scale"], s["branch_scale"]

    def inverse(v):
        return ((v ** 2).sum(1) / v.shape[1] + EPS) ** -0.5

    if op == "norm":
        r1 = inverse(x)
        z = s["residual"].double() * a + gate * post * x * r1.unsqueeze(1) * b
        v = z.to(t).double()  # the norm reads what is stored
        r2 = inverse(v)
        return z, v * pre * r2.unsqueeze(1), r1, r2
    n = case["cols"]
    r1, r2 = s["post_rstd"].double().unsqueeze(1), s["pre_rstd"].double().unsqueeze(1)
    zh = s["z"].double() * r2
    dpre = (s["dy"].double() * zh).sum(0)
    c = s["dy"].double() * pre
    dz = (c - zh * ((c * zh).sum(1, keepdim=True) / n)) * r2 + s["dz_add"].double()
    del zh, c
    xh = x * r1
    dp = dz * gate * b
    dpost = (dp * xh).sum(0)
    q = dp * post
    dx = (q - xh * ((q * xh).sum(1, keepdim=True) / n)) * r1
    out = dz * a, dx, dpost, dpre
    if case["gate"] == "none":
        return out
    dgate = dz * xh * post * b
    return out + (dgate.sum(0) if case["gate"] == "channel" else dgate,)
