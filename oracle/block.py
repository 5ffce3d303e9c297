"""Plain 64-bit definitions of the operators around the MLP (numpy): layer norm and its
gradients, dropout from Philox4x32-10, INT8 codes with one scale per row and their product.
Test infrastructure only; it shares no code with the library."""
from __future__ import annotations

import numpy as np

U64 = np.uint64
LOW = 0xFFFFFFFF


def philox4x32(counter, key, rounds: int = 10):
    """The four output words (uint64 arrays holding 32 bits) of Philox4x32 (Salmon, Moraes,
    Dror and Shaw, SC 2011): counter four arrays or numbers of 32 bits, key two."""
    c = [np.asarray(x, U64) for x in counter]
    k = [int(x) for x in key]
    for i in range(rounds):
        a, b = c[0] * U64(0xD2511F53), c[2] * U64(0xCD9E8D57)
        k0, k1 = (k[0] + i * 0x9E3779B9) & LOW, (k[1] + i * 0xBB67AE85) & LOW
        c = [(b >> U64(32)) ^ c[1] ^ U64(k0), b & U64(LOW),
             (a >> U64(32)) ^ c[3] ^ U64(k1), a & U64(LOW)]
    return c


def drop_numbers(row_index, cols: int, seed: int, offset: int) -> np.ndarray:
    """The 16-bit numbers of the elements of the given rows."""
    row_index = np.asarray(row_index, U64)
    blocks = (cols + 7) // 8
    c0 = np.tile(np.arange(blocks, dtype=U64), len(row_index))
    c1 = np.repeat(row_index, blocks)
    w = philox4x32((c0, c1, offset & LOW, (offset >> 32) & LOW), (seed & LOW, (seed >> 32) & LOW))
    n = np.stack([v for x in w for v in (x & U64(0xFFFF), x >> U64(16))], -1)
    return n.astype(np.int64).reshape(len(row_index), blocks * 8)[:, :cols]


def drop_factor(rows, cols: int, p: float, seed: int, offset: int) -> np.ndarray:
    """keep / (1 - p) of every element; rows a count or the rows' indices."""
    t = int(np.rint(float(np.float32(p)) * 65536.0))
    index = np.arange(rows) if np.isscalar(rows) else rows
    keep = drop_numbers(index, cols, seed, offset) >= t
    return np.where(keep, 65536.0 / (65536 - t) if t < 65536 else 0.0, 0.0)


def dropped(x, factor):
    """x times the factor, with +0 for a dropped element whatever x holds there."""
    with np.errstate(invalid="ignore"):
        return np.where(factor != 0.0, x * factor, 0.0)


def layer_norm(x, weight, bias, eps: float):
    """(y, mean, rstd) of float64 rows."""
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    return d * rstd[:, None] * weight + bias, mean, rstd


def layer_norm_backward(dy, z, weight, mean, rstd):
    """(dz, dweight, dbias)."""
    h = (z - mean[:, None]) * rstd[:, None]
    g = dy * weight
    dz = rstd[:, None] * (g - g.mean(1, keepdims=True) - h * (g * h).mean(1, keepdims=True))
    return dz, (dy * h).sum(0), dy.sum(0)


def quantize_int8(x):
    """(codes, scales) of float64 rows that hold binary32 values: 127 x is exact in 64 bits, and
    its quotient by the row's largest magnitude keeps its side of every border."""
    x = np.asarray(x, np.float64)
    top = np.abs(x).max(1)
    fine = np.isfinite(top) & (top > 0)
    q = np.rint(np.where(fine[:, None], x, 0.0) * 127.0 / np.where(fine, top, 1.0)[:, None])
    scale = np.where(np.isfinite(top), top / 127.0, np.nan)
    return q.astype(np.int8), scale


def int8_gemm(a, b, a_scale, b_scale, bias=None):
    """(y, the exact integer sums) with y in float64."""
    sums = (a.astype(np.float64) @ b.astype(np.float64).T)     # |sums| < 2^31: exact
    y = sums * a_scale[:, None] * b_scale
    return (y if bias is None else y + bias), sums
