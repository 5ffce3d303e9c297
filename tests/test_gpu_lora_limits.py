"""Adapters' weights that are not finite, and what they may touch (GPU)."""
import numpy as np
import pytest
import torch

import scaled_quantization_amd as sq
from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rank", [7, 16, 64])
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_weights_that_are_not_finite_touch_their_adapter_alone(t, rank):
    tokens, N, K, adapters = 150, 96, 136, 4
    g = torch.Generator().manual_seed(rank)
    rand = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).to(t)
    x, base = rand(tokens, K), rand(tokens, N)
    a, b = rand(adapters, rank, K, std=K ** -0.5), rand(adapters, N, rank, std=0.3)
    index = torch.randint(-1, adapters, (tokens,), generator=g, dtype=torch.int32)
    plan = torch.empty(sq.lora_plan_size(tokens, adapters), dtype=torch.int32, device=DEV)
    sq.lora_plan(index.to(DEV), adapters, plan)
    ws = torch.full((sq.lora_add_workspace(tokens, N, K, rank, adapters),), 255, dtype=torch.uint8, device=DEV)

    def run(a, b):
        y = torch.empty((tokens, N), dtype=t, device=DEV)
        sq.lora_add(x.to(DEV), a.to(DEV), b.to(DEV), torch.ones(adapters, device=DEV), plan, base.to(DEV), y, ws)
        return y.cpu()

    want = run(a, b)
    assert torch.isfinite(want).all()
    # a channel of b: that channel of the adapter's tokens
    bad = b.clone()
    bad[1, 5, rank - 1], bad[1, 40, 0] = float("inf"), float("nan")
    y, mine = run(a, bad), (index == 1).numpy()
    hit = np.zeros((tokens, N), dtype=bool)
    hit[np.ix_(mine, [5, 40])] = True
    hit = torch.from_numpy(hit)
    assert not torch.isfinite(y[hit]).any() and torch.equal(y[~hit], want[~hit])
    # a rank of a: all channels of the adapter's tokens
    bad = a.clone()
    bad[2, 3, 100] = float("nan")
    y, mine = run(bad, b), index == 2
    assert torch.isnan(y[mine]).all() and torch.equal(y[~mine], want[~mine])
