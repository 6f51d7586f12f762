"""Plain 64-bit references of the operators around dispatch and combine, from
their definitions (numpy, CPU), and the inputs their tests share.

e4m3 rows are held as the codes' bytes; values come from the format's closed
form, rounding from its steps.
"""
from __future__ import annotations

import numpy as np
import torch

from tests.fp8_checks import e4m3_values

BLOCK = 128
LUT = e4m3_values()
BF16_HALF = 2.0 ** -8           # half a step of bf16, relative
E4M3_HALF = 2.0 ** -4
FP32_HALF = 2.0 ** -24


def bf16(a) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def round_e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, ties to even, held to +-448."""
    a = np.maximum(np.abs(v), 2.0 ** -6)
    step = np.exp2(np.floor(np.log2(a)) - 3)
    return np.clip(np.round(v / step) * step, -448, 448)


def block_scale(v: np.ndarray):
    """(scale, inverse) of each block of 128, in 64 bits."""
    amax = np.abs(v.reshape(*v.shape[:-1], -1, BLOCK)).max(-1)
    small = amax < 448 * 2.0 ** -126
    scale = np.where(amax == 0, 1.0, np.where(small, 2.0 ** -126, amax / 448))
    with np.errstate(divide="ignore"):
        inv = np.where(amax == 0, 0.0, np.where(small, 2.0 ** 126, 448 / amax))
    return scale, inv


def coded(v: np.ndarray) -> np.ndarray:
    """The values that the codec's codes and scales stand for; inverse and
    product rounded to fp32, where the codec decides."""
    scale, inv = block_scale(v)
    inv = inv.astype(np.float32).astype(np.float64).repeat(BLOCK, -1)
    return round_e4m3((v * inv).astype(np.float32).astype(np.float64)) * scale.repeat(BLOCK, -1)


def rows_value(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    return LUT[q] * s.astype(np.float64).repeat(BLOCK, -1)


def weights_value(w: np.ndarray, s: np.ndarray) -> np.ndarray:
    n = w.shape[-2]
    return LUT[w] * s.astype(np.float64).repeat(BLOCK, -2)[..., :n, :].repeat(BLOCK, -1)


def make_rows(g, rows, k, spread=1.0):
    """Random finite codes and scales of different magnitude."""
    q = g.integers(0, 256, size=(rows, k), dtype=np.int64).astype(np.uint8)
    q[(q & 0x7F) == 0x7F] = 0x38
    s = np.exp(spread * g.standard_normal((rows, k // BLOCK))).astype(np.float32)
    return q, s


def make_weights(g, experts, n, k):
    q = g.integers(0, 256, size=(experts, n, k), dtype=np.int64).astype(np.uint8)
    q[(q & 0x7F) == 0x7F] = 0xB8
    s = (2.0 ** -12 * np.exp(g.standard_normal((experts, -(-n // BLOCK), k // BLOCK)))).astype(np.float32)
    return q, s


def product(x, xs, w, ws, offsets):
    """(y, bound): the grouped product in 64 bits, and for every output the
    sum over blocks of its largest |product|, which scales the error of the
    block sums."""
    rows, n = int(offsets[-1]), w.shape[1]
    y, big = np.zeros((rows, n)), np.zeros((rows, n))
    xv = rows_value(x[:rows], xs[:rows])
    for e in range(w.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        wv = weights_value(w[e], ws[e])
        y[a:b] = xv[a:b] @ wv.T
        for k0 in range(0, xv.shape[1], BLOCK):
            for r in range(a, b):
                big[r] += np.abs(xv[r, k0:k0 + BLOCK] * wv[:, k0:k0 + BLOCK]).max(-1)
    return y, big


def silu(v):
    return v / (1 + np.exp(-v))
