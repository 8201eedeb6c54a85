"""CPU oracle of the microscaled 4-bit format and the expert layer, in 64-bit floats from the definitions."""
from __future__ import annotations

import numpy as np

FP4_E4M3, FP4_E8M0 = 1, 2
FP4_BLOCK = {FP4_E4M3: 16, FP4_E8M0: 32}

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])
# the e4m3 numbers of bytes 0 .. 0x7e, and NaN
E4M3 = np.array([(b & 7) * 2.0 ** -9 if b < 8 else (1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 7) for b in range(127)] + [np.nan])


def fp4_scale_values(scales, fmt):
    scales = np.asarray(scales)
    if fmt == FP4_E4M3:
        return E4M3[scales]
    return np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))


def fp4_values(codes, scales, fmt, factor=1.0):
    """codes [rows, K] (0..15) and scale bytes [rows, K / block] -> float64 [rows, K]."""
    s = np.repeat(fp4_scale_values(scales, fmt), FP4_BLOCK[fmt], axis=-1)
    return E2M1[codes] * s * np.float64(factor)


def _nearest(v, grid):
    """Index of the grid's number nearest to v >= 0 (at most the last), ties to the even index."""
    i = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    lo, hi = v - grid[i - 1], grid[i] - v
    return np.where((lo < hi) | ((lo == hi) & (i % 2 == 1)), i - 1, i)


def fp4_quantize(x, fmt, factor=1.0):
    """fp16 [rows, K] -> (codes [rows, K], scale bytes [rows, K / block]); the factor is a number of 64 bits, as are the quotients
    that decide (6 factor and scale times factor are rounded to 64 bits before them)."""
    x = np.asarray(x, dtype=np.float16).astype(np.float64)
    rows, K = x.shape
    b = x.reshape(rows, -1, FP4_BLOCK[fmt])
    finite = np.isfinite(b).all(-1)
    b = np.where(finite[..., None], b, 0.0)
    a = np.abs(b).max(-1)
    f = np.float64(factor)
    if fmt == FP4_E4M3:
        byte = np.where(a > 0, np.maximum(_nearest(np.minimum(a / (6 * f), 448.0), E4M3[:127]), 1), 0)
        scale = E4M3[byte] * f
        nan = 0x7F
    else:
        e = np.where(a > 0, np.frexp(a)[1] - 3, -127)
        byte, scale, nan = e + 127, np.exp2(e.astype(np.float64)), 0xFF
    code = _nearest(np.minimum(np.abs(b) / np.where(scale > 0, scale, 1.0)[..., None], 6.0), E2M1[:8])
    code = np.where(finite[..., None], code + 8 * np.signbit(b), 0)
    return code.reshape(rows, K).astype(np.uint8), np.where(finite, byte, nan).astype(np.uint8)


def fp4_pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def fp4_unpack(packed):
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def fp4_tile(scales):
    """Scale bytes [rows, blocks] -> the tiles, zero where they reach over the matrix."""
    rows, blocks = scales.shape
    across = -(-blocks // 4)
    out = np.zeros((-(-rows // 128), across, 32, 4, 4), np.uint8)
    r, j = np.meshgrid(np.arange(rows), np.arange(blocks), indexing="ij")
    out[r // 128, j // 4, r % 32, r % 128 // 32, j % 4] = scales
    return out.reshape(-1)


def fp4_untile(tiles, rows, blocks):
    t = np.asarray(tiles).reshape(-(-rows // 128), -(-blocks // 4), 32, 4, 4)
    r, j = np.meshgrid(np.arange(rows), np.arange(blocks), indexing="ij")
    return t[r // 128, j // 4, r % 32, r % 128 // 32, j % 4]


def moe_route(logits, top_k, renorm):
    """(ids, weights) from logits [T, experts]: NaN counts as -infinity, ties go to the lowest index."""
    key = np.where(np.isnan(logits), -np.inf, logits)
    ids = np.argsort(-key, axis=-1, kind="stable")[:, :top_k]
    chosen = np.take_along_axis(logits, ids, -1)
    with np.errstate(all="ignore"):
        p = np.exp(chosen - chosen[:, :1])
        total = p.sum(-1, keepdims=True) if renorm else np.exp(logits - chosen[:, :1]).sum(-1, keepdims=True)
        return ids.astype(np.int32), p / total


def moe_activate(g, act):
    with np.errstate(over="ignore"):
        if act == 0:
            return g / (1 + np.exp(-g))
        return 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))
