"""Cases of the transformer-block operators around the MLP: layer norm and its backward pass,
dropout with the residual sum (alone, with the norm behind it, and backward), and the INT8
linear layer with one scale per token and one per output channel (alone, and behind a norm).

`run` computes them in elementary torch operations, or, where `own` is true, through
scaled_quantization_amd's entry points.

Formulas, with rows x cols inputs and statistics over a row:
  norm       mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps), y = (x - mu) rstd w + b
  norm_grad  g = dy w, h = (x - mu) rstd, dx = rstd (g - mean(g) - h mean(g h)),
             dw = sum over rows of dy h, db = sum over rows of dy
  dropout    keep(r, c) x(r, c) / (1 - p) + residual(r, c).  keep comes from Philox4x32-10 (Salmon,
             Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011): the
             block with key = seed and counter (c / 8, r, offset low, offset high) gives 8 numbers of
             16 bits, low half of a word first; element c takes number c % 8 and is kept when that
             is at least T = rint(65536 p); 1 - p is (65536 - T) / 65536
  linear     per token s = amax(x) / 127, q = rint(127 x / amax(x)), ties to even;
             y[m, n] = (sum over k of q[m, k] w8[n, k]) s[m] w_scale[n] + bias[n]
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the norm in front of a layer while one sequence decodes: latency
        {"name": "norm_one_token", "op": "norm", "rows": 1, "cols": 4096, "type": "bf16"},
        # 8 sequences x 2048 tokens of model width 768: the training benchmark's step
        {"name": "norm_train", "op": "norm", "rows": 16384, "cols": 768, "type": "bf16"},
        # the same step's backward pass
        {"name": "norm_grad_train", "op": "norm_grad", "rows": 16384, "cols": 768, "type": "bf16"},
        # ragged rows and an odd width: no row but the first is aligned
        {"name": "norm_grad_odd", "op": "norm_grad", "rows": 2049, "cols": 1001, "type": "f16"},
        # a wide model's backward pass, larger than every cache
        {"name": "norm_grad_wide", "op": "norm_grad", "rows": 65536, "cols": 4096, "type": "bf16"},
        # the tail of the MLP in training: dropout of the down-projection, residual sum, next norm
        {"name": "residual_train", "op": "residual", "rows": 16384, "cols": 768, "type": "bf16", "p": 0.1},
        # its backward pass at a wider model, ragged token count
        {"name": "residual_grad", "op": "residual_grad", "rows": 30001, "cols": 1600, "type": "bf16", "p": 0.1},
        # dropout and residual sum alone, in the type of a full-precision run, odd width
        {"name": "dropout_odd", "op": "dropout", "rows": 1023, "cols": 4097, "type": "f32", "p": 0.25},
        # one token of a decoding sequence through an INT8 layer: the weight's bytes and latency
        {"name": "linear_one_token", "op": "linear", "rows": 1, "n": 4096, "k": 4096, "type": "bf16"},
        # a decoding batch
        {"name": "linear_batch", "op": "linear", "rows": 48, "n": 4096, "k": 4096, "type": "f16"},
        # a prompt of ragged length and odd widths: norm, quantize, multiply
        {"name": "norm_linear_odd", "op": "norm_linear", "rows": 777, "n": 1023, "k": 1001, "type": "bf16"},
        # the fine-grained benchmark's layer: 65536 tokens
        {"name": "linear_large", "op": "linear", "rows": 65536, "n": 1024, "k": 4096, "type": "bf16"},
    ]


def _size(rng, low, high):
    """A whole number, spread over its logarithm; two of three are multiples of 8."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if v >= 16 and rng.random() < 0.67:
        v -= v % 8
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "residual", "residual_grad", "dropout", "linear",
                     "linear", "norm_linear"])
    case = {"op": op, "type": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op in ("linear", "norm_linear"):
        if op == "norm_linear" and case["type"] == "f32":
            # a norm in 32 bits moves some codes across a border: 32-bit outputs show each of them
            case["type"] = "bf16"
        case["rows"] = _size(rng, 1, 16384)
        case["n"] = _size(rng, 16, 8192)
        case["k"] = _size(rng, 16, 8192)
        return case
    case["cols"] = _size(rng, 64, 16384)
    case["rows"] = _size(rng, 1, min(65536, (1 << 25) // case["cols"]))
    if op in ("residual", "residual_grad", "dropout"):
        case["p"] = rng.choice([0.0625, 0.1, 0.25, 0.5])
    return case


def work(case):
    r, e = case["rows"], BYTES[case["type"]]
    if case["op"] in ("linear", "norm_linear"):
        n, k = case["n"], case["k"]
        norm = 2 * k * e if case["op"] == "norm_linear" else 0
        return {"bytes": r * k * e + n * k + r * n * e + 4 * n + n * e + norm, "flops": 2 * r * n * k}
    c = case["cols"]
    # tensors of rows x cols read and written, parameters, FP32 vectors of a row each
    tensors, params, stats = {"norm": (2, 2, 2), "norm_grad": (3, 1, 2), "residual": (4, 2, 2),
                              "residual_grad": (5, 1, 2), "dropout": (3, 0, 0)}[case["op"]]
    grads = 8 * c if case["op"].endswith("grad") else 0
    return {"bytes": tensors * r * c * e + params * c * e + 4 * stats * r + grads, "flops": 0}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t, r, op = TYPES[case["type"]], case["rows"], case["op"]

    def normal(*shape, std=1.0, mean=0.0, to=t):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(to)

    s = {"case": dict(case)}
    if op in ("linear", "norm_linear"):
        n, k = case["n"], case["k"]
        # activations have a few channels much larger than the rest
        channel = torch.where(torch.rand(k, generator=g, device="cuda") < 0.01, 12.0, 1.0)
        s["x"] = (torch.randn((r, k), generator=g, device="cuda") * channel).to(t)
        w = torch.randn((n, k), generator=g, device="cuda") * 0.02
        top = w.abs().amax(1)
        s["w8"] = torch.round(w * 127.0 / top[:, None]).to(torch.int8)
        s["w_scale"] = top / 127.0
        s["bias"] = normal(n, std=0.1)
        s["y"] = torch.empty((r, n), dtype=t, device="cuda")
        if op == "norm_linear":
            s["weight"], s["shift"] = normal(k, std=0.1, mean=1.0), normal(k, std=0.1)
            s["q"] = torch.empty((r, k), dtype=torch.int8, device="cuda")
            s["q_scale"] = torch.empty(r, dtype=torch.float32, device="cuda")
        # codes and scales of the tokens, and 16 MiB for a product split over k
        s["workspace"] = torch.empty(r * (k + 16) + 4 * r + 1024 + (16 << 20), dtype=torch.uint8,
                                     device="cuda")
        return s
    c = case["cols"]
    s["x"] = normal(r, c, std=1.5, mean=0.25)
    if op == "dropout":
        s["residual"] = normal(r, c)
    if op == "residual":
        s["residual"] = normal(r, c, std=2.0)
    if op != "dropout":
        s["weight"], s["bias"] = normal(c, std=0.1, mean=1.0), normal(c, std=0.1)
    if "p" in case:
        s["rng"] = torch.tensor([seed * 7919 + 12345678901234, (seed << 33) + 5], dtype=torch.int64,
                                device="cuda")
    if op.endswith("grad"):
        s["dy"] = normal(r, c, std=0.02)
        x = s["x"].float()
        s["mean"] = x.mean(1)
        s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + EPS)
        if op == "residual_grad":
            s["dz_add"] = normal(r, c, std=0.02)
            s["dx"] = torch.empty_like(s["x"])
        s["dz"] = torch.empty_like(s["x"])
        s["dweight"] = torch.empty(c, dtype=torch.float32, device="cuda")
        s["dbias"] = torch.empty_like(s["dweight"])
        s["workspace"] = torch.empty(2 * min(r, 1024) * c, dtype=torch.float32, device="cuda")
    else:
        s["out"] = torch.empty_like(s["x"])
        if op != "dropout":
            s["z"] = torch.empty_like(s["x"])
            s["mean"] = torch.empty(r, dtype=torch.float32, device="cuda")
            s["rstd"] = torch.empty_like(s["mean"])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import scaled_quantization_amd as sq
    case = s["case"]
    op = case["op"]
    if op == "norm":
        sq.layer_norm(s["x"], s["weight"], s["bias"], EPS, s["out"], s["mean"], s["rstd"])
        return s["out"], s["mean"], s["rstd"]
    if op == "norm_grad":
        sq.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dz"],
                               s["dweight"], s["dbias"], s["workspace"])
        return s["dz"], s["dweight"], s["dbias"]
    if op == "residual":
        sq.dropout_add_layer_norm(s["x"], s["residual"], case["p"], s["rng"], s["weight"], s["bias"],
                                  EPS, s["z"], s["out"], s["mean"], s["rstd"])
        return s["z"], s["out"], s["mean"], s["rstd"]
    if op == "residual_grad":
        sq.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dz"],
                               s["dweight"], s["dbias"], s["workspace"], s["dz_add"], case["p"],
                               s["rng"], s["dx"])
        return s["dz"], s["dx"], s["dweight"], s["dbias"]
    if op == "dropout":
        sq.dropout_add(s["x"], s["residual"], case["p"], s["rng"], s["out"])
        return s["out"]
    if op == "linear":
        sq.int8_linear(s["x"], s["w8"], s["w_scale"], s["y"], s["workspace"], s["bias"])
        return s["y"]
    sq.layer_norm_quantize_int8(s["x"], s["weight"], s["shift"], EPS, s["q"], s["q_scale"])
    sq.int8_gemm(s["q"], s["w8"], s["q_scale"], s["w_scale"], s["y"], s["bias"], s["workspace"])
    return s["y"]


def _mask(rows, cols, p, rng):
    """keep as a [rows, cols] truth value, and 1 / (1 - p)."""
    low = 0xFFFFFFFF
    t = round(float(np.float32(p)) * 65536)
    blocks = (cols + 7) // 8
    c0 = torch.arange(blocks, device="cuda").expand(rows, blocks)
    c1 = torch.arange(rows, device="cuda")[:, None].expand(rows, blocks)
    seed, offset = rng[0], rng[1]
    c2, c3 = offset & low, (offset >> 32) & low
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], -1)
    numbers = torch.stack([words & 0xFFFF, words >> 16], -1).reshape(rows, blocks * 8)[:, :cols]
    return numbers >= t, (65536 / (65536 - t) if t < 65536 else 0.0)


def _dropped(x, p, rng):
    keep, scale = _mask(x.shape[0], x.shape[1], p, rng)
    return torch.where(keep, x * scale, 0.0)


def _norm(x, weight, bias):
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + EPS)
    return d * rstd[:, None] * weight.float() + bias.float(), mean, rstd


def _multiplied(x, s):
    """The INT8 linear layer of activations x.  127 x and the quotient's side of a border are exact
    in 32 bits for values of 16 bits; those of 32 bits come in 64."""
    top = x.abs().amax(1)
    q = torch.round(x * 127.0 / torch.where(top > 0, top, 1.0)[:, None]).float()
    top = top.float()
    y = (q @ s["w8"].float().t()) * (top / 127.0)[:, None] * s["w_scale"]
    return (y + s["bias"].float()).to(s["y"].dtype)


def _plain(s):
    case = s["case"]
    op, t = case["op"], s["x"].dtype
    x = s["x"].float()
    if op == "norm":
        y, mean, rstd = _norm(x, s["weight"], s["bias"])
        return y.to(t), mean, rstd
    if op == "residual":
        z = (s["residual"].float() + _dropped(x, case["p"], s["rng"])).to(t)
        y, mean, rstd = _norm(z.float(), s["weight"], s["bias"])
        return z, y.to(t), mean, rstd
    if op == "dropout":
        return (s["residual"].float() + _dropped(x, case["p"], s["rng"])).to(t)
    if op in ("norm_grad", "residual_grad"):
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        h = (x - s["mean"][:, None]) * rstd
        g = dy * s["weight"].float()
        dz = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
        dweight, dbias = (dy * h).sum(0), dy.sum(0)
        if op == "norm_grad":
            return dz.to(t), dweight, dbias
        dz = dz + s["dz_add"].float()
        return dz.to(t), _dropped(dz, case["p"], s["rng"]).to(t), dweight, dbias
    if op == "linear":
        return _multiplied(x.double() if t == torch.float32 else x, s)
    return _multiplied(_norm(x, s["weight"], s["shift"])[0], s)


# ------------------------------------------------------------------ 64 bits
def _philox(rows, cols, rng):
    """The 16-bit numbers of every element, as numpy."""
    u = np.uint64
    blocks = (cols + 7) // 8
    seed, offset = (int(v) & (2**64 - 1) for v in rng.tolist())
    x = [np.tile(np.arange(blocks, dtype=u), rows), np.repeat(np.arange(rows, dtype=u), blocks),
         np.full(rows * blocks, offset & 0xFFFFFFFF, u), np.full(rows * blocks, offset >> 32, u)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for i in range(10):
        p0, p1 = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        ka, kb = (key[0] + i * 0x9E3779B9) % 2**32, (key[1] + i * 0xBB67AE85) % 2**32
        x = [(p1 >> u(32)) ^ x[1] ^ u(ka), p1 & u(0xFFFFFFFF),
             (p0 >> u(32)) ^ x[3] ^ u(kb), p0 & u(0xFFFFFFFF)]
    out = np.empty((rows * blocks, 8), np.int32)
    for w in range(4):
        out[:, 2 * w] = (x[w] & u(0xFFFF)).astype(np.int32)
        out[:, 2 * w + 1] = (x[w] >> u(16)).astype(np.int32)
    return out.reshape(rows, blocks * 8)[:, :cols]


def exact(case, seed):
    """The definitions in 64 bits, on the GPU but for the random numbers."""
    if "p" in case and case["rows"] * case["cols"] > 1 << 26:
        return None
    s = prepare(case, seed)
    op, t = case["op"], s["x"].dtype
    x = s["x"].double()
    if "p" in case:
        t16 = round(float(np.float32(case["p"])) * 65536)
        numbers = torch.from_numpy(_philox(case["rows"], case["cols"], s["rng"])).cuda()
        factor = (numbers >= t16).double() * (65536.0 / (65536 - t16))

    def moments(v):
        mean = v.sum(1) / v.shape[1]
        variance = ((v - mean.unsqueeze(1)) ** 2).sum(1) / v.shape[1]
        return mean, (variance + EPS) ** -0.5

    if op == "dropout":
        return s["residual"].double() + x * factor
    if op in ("norm", "norm_linear"):
        mean, rstd = moments(x)
        shift = s["bias" if op == "norm" else "shift"].double()
        y = (x - mean.unsqueeze(1)) * rstd.unsqueeze(1) * s["weight"].double() + shift
        if op == "norm":
            return y, mean, rstd
        x = y
    if op == "residual":
        z = s["residual"].double() + x * factor
        v = z.to(t).double()  # the norm reads what is stored
        mean, rstd = moments(v)
        y = (v - mean.unsqueeze(1)) * rstd.unsqueeze(1) * s["weight"].double() + s["bias"].double()
        return z, y, mean, rstd
    if op in ("norm_grad", "residual_grad"):
        rstd = s["rstd"].double().unsqueeze(1)
        h = (x - s["mean"].double().unsqueeze(1)) * rstd
        del x
        dy = s["dy"].double()
        dweight, dbias = (dy * h).sum(0), dy.sum(0)
        g = dy * s["weight"].double()
        del dy
        a, b = g.sum(1, keepdim=True), (g * h).sum(1, keepdim=True)
        dz = (g - (a + h * b) / case["cols"]) * rstd
        if op == "norm_grad":
            return dz, dweight, dbias
        dz = dz + s["dz_add"].double()
        return dz, dz * factor, dweight, dbias
    top = x.abs().max(1).values.unsqueeze(1)
    q = (x * 127.0 / top.clamp(min=1e-300)).round()
    sums = torch.matmul(q, s["w8"].double().t().contiguous())
    return sums * (top / 127.0) * s["w_scale"].double() + s["bias"].double()
