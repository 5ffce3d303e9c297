"""Low-rank adapters of many requests on the GPU, against their 64-bit definition (oracle/gated.py).

Tolerance, from the arithmetic: the product a x goes through matrix instructions (K / 16 + 48 roundings of a term
at most, 2 U each where an instruction truncates, U = 2^-24) and up to 16 partial sums; its value is then held
as two 16-bit numbers, off by half a step of the type twice, H^2 (bf16 2^-16, fp16 2^-22; the smaller part of fp16
may be a subnormal, 2^-25 of the row's largest); the product with b has (2 R / 16 + 48) such roundings; scale,
sum and the last rounding follow.  All are relative to |scale| |b| |a| |x|; the subnormal
part to the row's largest |a x|, which |scale| sum |b| carries.
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


def half(t):
    return torch.finfo(t).eps / 2


def draw(shape, t, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(t)


def f64(x):
    return x.cpu().double().numpy()


def indexes(kind, tokens, adapters, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "none":
        return np.full(tokens, -1)
    if kind == "one":
        return np.full(tokens, adapters - 1)
    if kind == "packed":
        return np.sort(rng.integers(-1, adapters, tokens))[::-1].copy()
    return rng.integers(-1, adapters, tokens)


def make_plan(index, adapters):
    plan = torch.full((sq.lora_plan_size(len(index), adapters),), -7, dtype=torch.int32, device=DEV)
    sq.lora_plan(torch.from_numpy(index).to(torch.int32).to(DEV), adapters, plan)
    return plan


def workspace(tokens, N, K, rank, adapters):
    return torch.full((sq.lora_add_workspace(tokens, N, K, rank, adapters),), 255, dtype=torch.uint8, device=DEV)


def inputs(tokens, N, K, rank, adapters, t, seed=0):
    g = torch.Generator().manual_seed(seed + 9)
    return (draw((tokens, K), t, seed), draw((adapters, rank, K), t, seed + 1, K ** -0.5),
            draw((adapters, N, rank), t, seed + 2, 0.3), 0.25 + 2 * torch.rand(adapters, generator=g))


def check(x, a, b, scale, index, base, ranks, y, t, what):
    fx, fa, fb, fs = f64(x), f64(a), f64(b), f64(scale)
    fbase = np.zeros(y.shape) if base is None else f64(base)
    r = None if ranks is None else ranks.numpy()
    if r is not None:      # what unused ranks hold does not matter
        fa, fb = np.nan_to_num(fa, nan=0.0), np.nan_to_num(fb, nan=0.0)
    ref, size = OG.lora_add(fx, fa, fb, fs, index, fbase, r)
    K, R = fx.shape[1], fa.shape[1]
    off = size * ((K / 16 + 64 + R / 8 + 48) * 2 * U + half(t) ** 2)
    if t == F16:
        for tok, i in enumerate(index):
            if 0 <= i < len(fa):
                off[tok] += 2.0 ** -24 * abs(fs[i]) * np.abs(fb[i]).sum(1) * np.abs(fa[i] @ fx[tok]).max()
    off += 2 * U * (np.abs(ref) + np.abs(fbase))
    tol = off + half(t) * (np.abs(ref) + off) + 2.0 ** -25
    got = f64(y)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}: {got[bad][0]} for "
                           f"{ref[bad][0]}, allowed {tol[bad][0]}")
    none = ~((index >= 0) & (index < len(fa)))
    assert np.array_equal(got[none], fbase[none]), what + ": tokens without an adapter"


def case(tokens, N, K, rank, adapters, t, kind="mixed", ragged=False, in_place=False, base=True, seed=0):
    x, a, b, scale = inputs(tokens, N, K, rank, adapters, t, seed)
    index = indexes(kind, tokens, adapters, seed)
    ranks = None
    if ragged:
        ranks = torch.from_numpy(np.random.default_rng(3).integers(-1, rank + 2, adapters)).to(torch.int32)
        for i, r in enumerate(ranks.tolist()):
            a[i, max(r, 0):], b[i, :, max(r, 0):] = float("nan"), float("nan")
    add = draw((tokens, N), t, seed + 5) if base else None
    y = add.to(DEV) if in_place else torch.full((tokens, N), float("nan"), dtype=t, device=DEV)
    from_ = y if in_place else None if add is None else add.to(DEV)
    plan = make_plan(index, adapters)
    sq.lora_add(x.to(DEV), a.to(DEV), b.to(DEV), scale.to(DEV), plan, from_, y,
                workspace(tokens, N, K, rank, adapters), None if ranks is None else ranks.to(DEV))
    check(x, a, b, scale, index, add, ranks, y, t, f"{tokens} {N} {K} {rank} {adapters} {kind}")


# ------------------------------------------------------------------ plan
@pytest.mark.parametrize("tokens, adapters", [(1, 1), (5, 3), (63, 2), (64, 64), (65, 1), (1000, 7), (1024, 2048),
                                              (1025, 900), (5003, 8), (70000, 33), (300000, 2000)])
@pytest.mark.parametrize("kind", ["mixed", "packed", "one", "none"])
def test_plan(tokens, adapters, kind):
    index = indexes(kind, tokens, adapters, tokens)
    # adapters out of range are none
    if kind == "mixed" and tokens > 4:
        index[1], index[3] = adapters, -2 ** 31
    plan = make_plan(index, adapters).cpu().numpy()
    tiles, tok, ad, zero = plan[:4]
    assert (tok, ad, zero) == (tokens, adapters, 0)
    group = np.where((index >= 0) & (index < adapters), index, adapters)
    order = plan[4:4 + tokens]
    assert np.array_equal(order, np.argsort(group, kind="stable"))
    entry = plan[4 + tokens:].reshape(-1, 2)
    assert tiles <= len(entry)
    start, adapter, count = entry[:tiles, 0], entry[:tiles, 1] >> 8, entry[:tiles, 1] & 255
    assert (count >= 1).all() and (count <= 32).all()
    assert np.array_equal(start, np.concatenate([[0], np.cumsum(count)[:-1]])) and count.sum() == tokens
    assert np.array_equal(np.repeat(np.where(adapter < 0, adapters, adapter), count), group[order])
    # as few tiles as the groups allow
    assert tiles == sum(-(-c // 32) for c in np.unique(group, return_counts=True)[1])


# ------------------------------------------------------------------ sums
@pytest.mark.parametrize("t", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 64, 64, 8, 1), (1, 4096, 4096, 16, 3), (3, 33, 100, 1, 2), (17, 512, 256, 16, 17),
                                   (64, 700, 1000, 16, 64), (64, 96, 130, 7, 5), (40, 513, 72, 20, 2),
                                   (200, 130, 520, 64, 3), (100, 8, 8, 128, 4), (65, 1, 1, 3, 2),
                                   (33, 40, 4100, 256, 2), (500, 1030, 64, 33, 9)], ids=lambda s: "x".join(map(str, s)))
def test_shapes(shape, t):
    case(*shape, t)
    case(*shape, t, ragged=True, kind="packed", in_place=True, seed=1)


@pytest.mark.parametrize("kind", ["mixed", "packed", "one", "none"])
def test_orders_and_bases(kind):
    case(100, 200, 136, 16, 6, BF16, kind)
    case(100, 200, 136, 16, 6, BF16, kind, base=False)
    case(100, 201, 137, 16, 6, F16, kind, in_place=True)


def test_many_tokens():
    case(6000, 96, 128, 16, 5, BF16, "packed")
    case(6000, 64, 64, 8, 300, F16)


def test_more_tiles_than_a_grid_dimension():
    tokens, N, K, rank = 32 * 32768 + 77, 8, 8, 3
    x, a, b, scale = inputs(tokens, N, K, rank, 1, BF16)
    base = draw((tokens, N), BF16, 5)
    index = np.zeros(tokens, dtype=np.int64)
    index[-60:] = -1
    y = torch.full((tokens, N), float("nan"), dtype=BF16, device=DEV)
    sq.lora_add(*(v.to(DEV) for v in (x, a, b, scale)), make_plan(index, 1), base.to(DEV), y,
                workspace(tokens, N, K, rank, 1))
    fx, fa, fb, fbase, fs = (v.double() for v in (x, a[0], b[0], base, scale[0]))
    ref, size = fbase + fs * (fx @ fa.t()) @ fb.t(), fs * (fx.abs() @ fa.abs().t()) @ fb.abs().t()
    ref[-60:], size[-60:] = fbase[-60:], 0.0
    off = size * ((K / 16 + 64 + rank / 8 + 48) * 2 * U + half(BF16) ** 2) + 2 * U * (ref.abs() + fbase.abs())
    assert ((y.cpu().double() - ref).abs() <= off + half(BF16) * (ref.abs() + off) + 2.0 ** -25).all()
    assert torch.equal(y[-60:].cpu(), base[-60:])


def test_one_plan_for_layers_of_other_sizes():
    tokens, adapters = 90, 4
    index = indexes("mixed", tokens, adapters, 2)
    plan = make_plan(index, adapters)
    for N, K, rank in ((64, 128, 8), (256, 64, 32), (72, 200, 8)):
        x, a, b, scale = inputs(tokens, N, K, rank, adapters, BF16, N)
        y = torch.empty((tokens, N), dtype=BF16, device=DEV)
        sq.lora_add(*(v.to(DEV) for v in (x, a, b, scale)), plan, None, y, workspace(tokens, N, K, rank, adapters))
        check(x, a, b, scale, index, None, None, y, BF16, "shared plan")


def test_plan_of_other_sizes_writes_nothing():
    tokens, adapters = 90, 4
    x, a, b, scale = (v.to(DEV) for v in inputs(tokens, 64, 64, 8, adapters, BF16))
    good = make_plan(indexes("mixed", tokens, adapters), adapters)
    plan = torch.zeros_like(good)
    other = make_plan(indexes("mixed", 50, 7), 7)
    plan[:min(len(other), len(plan))] = other[:len(plan)]
    for p in (plan, torch.zeros_like(good), torch.full_like(good, -1)):
        y = torch.full((tokens, 64), 3.0, dtype=BF16, device=DEV)
        sq.lora_add(x, a, b, scale, p, None, y, workspace(tokens, 64, 64, 8, adapters))
        assert (y == 3).all()


def test_large_and_small_products_keep_their_size():
    # a x past fp16's range, and far below it, with a scale that brings it back
    tokens, N, K, rank, adapters = 40, 64, 64, 16, 3
    for factor in (2.0 ** 12, 2.0 ** -12):
        x, a, b, scale = inputs(tokens, N, K, rank, adapters, F16)
        x, a = (x.float() * factor).half(), (a.float() * (2.0 ** 6 if factor > 1 else 2.0 ** -2)).half()
        scale = scale / factor
        index = indexes("mixed", tokens, adapters)
        y = torch.empty((tokens, N), dtype=F16, device=DEV)
        sq.lora_add(*(v.to(DEV) for v in (x, a, b, scale)), make_plan(index, adapters), None, y,
                    workspace(tokens, N, K, rank, adapters))
        check(x, a, b, scale, index, None, None, y, F16, f"factor {factor}")


def test_tokens_that_are_not_finite_touch_no_other():
    tokens, N, K, rank, adapters = 50, 64, 136, 16, 3
    x, a, b, scale = inputs(tokens, N, K, rank, adapters, BF16)
    index = indexes("one", tokens, adapters)
    x[2, 5], x[40, 100] = float("nan"), float("inf")
    y = torch.empty((tokens, N), dtype=BF16, device=DEV)
    sq.lora_add(*(v.to(DEV) for v in (x, a, b, scale)), make_plan(index, adapters), None, y,
                workspace(tokens, N, K, rank, adapters))
    keep = [i for i in range(tokens) if i not in (2, 40)]
    assert torch.isfinite(y[keep]).all() and not torch.isfinite(y[[2, 40]]).any()


def test_at_any_alignment():
    tokens, N, K, rank, adapters, t = 70, 65, 128, 16, 3, BF16
    host = inputs(tokens, N, K, rank, adapters, t)
    x, a, b = (torch.empty(v.numel() + 1, dtype=t, device=DEV) for v in host[:3])
    args = []
    for room, v in zip((x, a, b), host):
        room[1:] = v.reshape(-1).to(DEV)
        args.append(room[1:].view(v.shape))
    index = indexes("mixed", tokens, adapters)
    base = draw((tokens, N), t, 4)
    room = torch.full((tokens * N + 2,), 7.0, dtype=t, device=DEV)
    y = room[1:-1].view(tokens, N)
    y.copy_(base.to(DEV))
    sq.lora_add(*args, host[3].to(DEV), make_plan(index, adapters), y, y, workspace(tokens, N, K, rank, adapters))
    check(*host, index, base, None, y, t, "offset")
    assert room[0] == 7 and room[-1] == 7


def test_captured_with_its_plan_and_replayed():
    tokens, N, K, rank, adapters, t = 300, 264, 512, 16, 6, BF16
    x, a, b, scale = (v.to(DEV) for v in inputs(tokens, N, K, rank, adapters, t))
    index = torch.zeros(tokens, dtype=torch.int32, device=DEV)
    plan = torch.empty(sq.lora_plan_size(tokens, adapters), dtype=torch.int32, device=DEV)
    base, y = draw((tokens, N), t, 8).to(DEV), torch.empty((tokens, N), dtype=t, device=DEV)
    ws = workspace(tokens, N, K, rank, adapters)

    def step():
        sq.lora_plan(index, adapters, plan)
        sq.lora_add(x, a, b, scale, plan, base, y, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        index.copy_(torch.from_numpy(indexes("mixed", tokens, adapters, seed)).to(torch.int32))
        y.fill_(float("nan"))
        plan.fill_(-1)
        ws.fill_(255)
        graph.replay()
        got = y.clone()
        torch.cuda.synchronize()
        step()
        assert torch.equal(got, y)
        check(x, a, b, scale, index.cpu().numpy(), base, None, y, t, "replay")
