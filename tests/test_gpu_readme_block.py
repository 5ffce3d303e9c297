"""README's example of the operators around the MLP runs as written (GPU), against the 64-bit definitions
(oracle/block.py) with the tolerances of test_gpu_block_norm and test_gpu_int8."""
import os
import re

import numpy as np
import pytest
import torch

import oracle.block as OB
from gpu_util import DEV
from test_gpu_block_norm import U, check_backward, check_norm, close, draw, f64, half, tiny
from test_gpu_int8 import check_product

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_block_example():
    blocks = re.findall(r"```py\n(.*?)```", open(README).read(), re.S)
    assert len(blocks) == 1
    t, shape = torch.bfloat16, (2048, 768)
    cpu = {"x": draw(shape, t, 1), "residual": draw(shape, t, 2, 2.0), "dy": draw(shape, t, 3),
           "dz_next": draw(shape, t, 4), "weight": draw(768, t, 5, 0.1, 1.0), "bias": draw(768, t, 6),
           "w": draw((1024, 768), t, 7, 0.02)}
    ns = {k: v.to(DEV) for k, v in cpu.items()}
    exec(blocks[0], ns)
    torch.cuda.synchronize()
    f = OB.drop_factor(*shape, 0.1, 1234, 7 * 12 + 3)
    x, res, w, b = (f64(cpu[k]) for k in ("x", "residual", "weight", "bias"))
    z = x * f + res
    close(ns["z"], z, 2 * U * (np.abs(x * f) + np.abs(z)) * (1 + half(t)) + half(t) * np.abs(z) + tiny(t), "z")
    check_norm(f64(ns["z"]), w, b, 1e-5, ns["y"], ns["mean"], ns["rstd"], t, "norm")
    check_backward(ns["dy"], ns["z"], ns["weight"], ns["mean"], ns["rstd"], ns["dz_next"], ns["dz"], ns["dx"],
                   ns["dweight"], ns["dbias"], t, "backward", f)
    w8, s = OB.quantize_int8(f64(cpu["w"]))
    assert np.array_equal(ns["w8"].cpu().numpy(), w8)
    close(ns["w_scale"], s, U * s, "weight scale")
    w_scale = f64(ns["w_scale"]).astype(np.float32)
    q, s = OB.quantize_int8(f64(ns["y"]))
    check_product(ns["up"], q, w8, s.astype(np.float32), w_scale, None, t, "linear")
    check_product(ns["up8"], ns["q"].cpu().numpy(), w8, f64(ns["q_scale"]).astype(np.float32), w_scale, None, t,
                  "product behind the norm")
    z8 = x + res
    close(ns["z8"], z8, U * np.abs(z8) + half(t) * np.abs(z8) + tiny(t), "z8")
