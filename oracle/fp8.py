"""fp64 references of the residual RMS norm, of 8-bit matrices with a scale per
block of 128, and of their product."""
from __future__ import annotations

import numpy as np

FP8_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100


def e4m3(x):
    """x rounded to the nearest e4m3 value (ties to even), clamped to +-448."""
    x = np.clip(np.asarray(x, np.float64), -FP8_MAX, FP8_MAX)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.abs(x)))
    e = np.where(np.isfinite(e), np.maximum(e, -6.0), -6.0)
    step = 2.0 ** (e - 3.0)
    return np.round(x / step) * step


def block_max(x, block_rows):
    """Largest magnitude per block of block_rows x 128: [ceil(K/128), blocks of rows]."""
    x = np.abs(np.asarray(x, np.float64))
    R, K = x.shape
    out = np.zeros((-(-K // 128), -(-R // block_rows)))
    for kb in range(out.shape[0]):
        for rb in range(out.shape[1]):
            out[kb, rb] = x[rb * block_rows:(rb + 1) * block_rows,
                            kb * 128:(kb + 1) * 128].max(initial=0.0)
    return out


def spread(v, block_rows, R, K):
    """Block values [ceil(K/128), blocks of rows] for each element of [R, K]."""
    return np.asarray(v, np.float64).T.repeat(block_rows, 0)[:R].repeat(128, 1)[:, :K]


def quantize(x, block_rows):
    """(values of the codes [R, K], scale) of x [R, K]."""
    amax = np.maximum(block_max(x, block_rows), AMAX_FLOOR)
    f = spread(FP8_MAX / amax, block_rows, *np.shape(x))
    return e4m3(np.asarray(x, np.float64) * f), amax / FP8_MAX


def dequantize(codes, scale, block_rows):
    codes = np.asarray(codes, np.float64)
    return codes * spread(scale, block_rows, *codes.shape)


def matmul(a, a_scale, b, b_scale, b_block_rows):
    return dequantize(a, a_scale, 1) @ dequantize(b, b_scale, b_block_rows).T


def rms_norm(s, w, eps):
    s = np.asarray(s, np.float64)
    return s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)


def rms_norm_bwd(s, w, dy, dsum, eps):
    """(dx, dw)."""
    s, w, dy = (np.asarray(v, np.float64) for v in (s, w, dy))
    r = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    wdy = w * dy
    dx = r * (wdy - s * r * r * (s * wdy).mean(-1, keepdims=True))
    if dsum is not None:
        dx = dx + np.asarray(dsum, np.float64)
    return dx, (dy * s * r).sum(0)
