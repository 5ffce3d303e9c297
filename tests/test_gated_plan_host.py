"""Which kernel each size of tests/gated_shapes.py reaches on a device of 256 compute units, from the library's own
plan, built for the host (csrc/product_plan.hpp is plain C++)."""
import ctypes
import os
import shutil
import subprocess

import pytest

import gated_shapes as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUS = 256


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plan")
    src, so = d / "plan.cpp", d / "plan.so"
    src.write_text('#include "product_plan.hpp"\n'
                   'extern "C" void plan(long long m, long long n, long long stages, int dual, double cus, int* out) {\n'
                   '  const auto p = fp8dp::plan_product(m, n, stages, dual, true, cus);\n'
                   '  out[0] = p.shape; out[1] = p.splits; out[2] = (int)fp8dp::tiles_of(p.shape, m, n);\n}\n')
    subprocess.run([cc, "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(ROOT, "scaled_quantization_amd", "csrc"),
                    str(src), "-o", str(so)], check=True)
    f = ctypes.CDLL(str(so)).plan
    f.argtypes = [ctypes.c_longlong] * 3 + [ctypes.c_int, ctypes.c_double, ctypes.c_void_p]
    f.restype = None

    def key(m, n, stages, dual):
        out = (ctypes.c_int * 3)()
        f(m, n, stages, dual, CUS, out)
        shape, splits, tiles = out
        pieces = tiles * splits
        slots = 4 if shape == 2 and pieces <= CUS else 2     # small tiles: four where each has a compute unit
        grid = CUS * (2 if shape == 2 and slots == 2 else 1)
        return (("256", "192", "128")[shape], slots, splits > 1, pieces > grid), stages // splits
    return key


def up(v):
    return -(-v // 64)


PRODUCTS = {"forward": lambda M, N, K: (M, 2 * N, up(K), 1), "dx": lambda M, N, K: (M, K, 2 * up(N), 0),
            "dw": lambda M, N, K: (128 * up(N), K, up(M), 0)}


@pytest.mark.parametrize("which, table", [("forward", S.FORWARD), ("dx", S.DX), ("dw", S.DW)])
def test_sizes_reach_their_kernels(plan, which, table):
    for want, (M, N, K) in table.items():
        got, stages = plan(*PRODUCTS[which](M, N, K))
        assert got == want and stages >= 5, (which, M, N, K, got, stages)
        assert K % 8 == 0 and {"forward": K, "dx": N, "dw": M}[which] % 64 != 0


def test_padded_sizes_are_copied_and_reach_large_tiles(plan):
    for which, (M, N, K) in S.PADDED.items():
        assert K % 8 != 0 and M * N * K >= 256e6
        assert plan(*PRODUCTS[which](M, N, K))[0][0] in ("192", "256")
