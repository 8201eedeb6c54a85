"""CPU oracle of the paged KV cache: rotary positions, cache append, attention.

Plain numpy from the definitions in include/exq.h: positions and turns in
Python integers, cos and sin in float64 rounded once to float32, attention in
float64. Shares no code with the library.
"""
from __future__ import annotations

import numpy as np

from .exq_oracle import kv_dequantize, kv_pack, kv_quantize, kv_unpack  # noqa: F401

TWO_PI = 2.0 * np.pi


def rope_freqs(R, base=10000.0, scaling=0, factor=1.0, orig_ctx=0.0, low=1.0, high=32.0):
    """(radians per position [R/2], gain) for the scalings none, linear, NTK, ramp over pairs, bands (0 .. 4)."""
    j = np.arange(R // 2, dtype=np.float64)
    if scaling == 2:
        base = base * factor ** (R / (R - 2))
    f = base ** (-2.0 * j / R)
    gain = 1.0
    if scaling == 1:
        f = f / factor
    elif scaling == 3:
        def pair(turns):
            return R * np.log(orig_ctx / (turns * TWO_PI)) / (2 * np.log(base))
        a, b = max(np.floor(pair(high)), 0), min(np.ceil(pair(low)), R - 1)
        stretched = np.clip((j - a) / max(b - a, 1e-3), 0, 1)
        f = f / factor * stretched + f * (1 - stretched)
        gain = 0.1 * np.log(factor) + 1 if factor > 1 else 1.0
    elif scaling == 4:
        m = np.clip((orig_ctx * f / TWO_PI - low) / (high - low), 0, 1)
        f = (1 - m) * f / factor + m * f
    return f, gain


def rope_steps(f):
    """Turns per position in units of 2^-64, uint64."""
    out = []
    for x in np.asarray(f, dtype=np.float64):
        t = x / TWO_PI
        out.append(int(np.rint(np.ldexp(t - np.floor(t), 64))) % (1 << 64))
    return np.array(out, dtype=np.uint64)


def rope_cos_sin(steps, pos, gain=1.0):
    """float32 [tokens, R/2] of gain cos, gain sin of 2 pi frac(pos step / 2^64)."""
    c = np.empty((len(pos), len(steps)), dtype=np.float32)
    s = np.empty_like(c)
    for i, p in enumerate(np.asarray(pos).tolist()):
        for j, st in enumerate(np.asarray(steps).tolist()):
            turn = (int(p) * int(st)) % (1 << 64)
            quarter, rest = (turn + (1 << 61)) >> 62, 0
            rest = turn - (quarter << 62)                       # at most an eighth of a turn either way
            x = TWO_PI * (rest / 2.0 ** 64)
            cc, ss = [(np.cos(x), np.sin(x)), (-np.sin(x), np.cos(x)), (-np.cos(x), -np.sin(x)),
                      (np.sin(x), -np.cos(x))][quarter % 4]
            c[i, j], s[i, j] = np.float32(cc * gain), np.float32(ss * gain)
    return c, s


def rope(x, steps, pos, R, interleaved=False, gain=1.0, grad=False):
    """fp16 [tokens, heads, D] turned; products, sums and the result each rounded to nearest."""
    c, s = (t[:, None, :] for t in rope_cos_sin(steps, pos, gain))
    s = -s if grad else s
    y = np.array(x, dtype=np.float16)
    f = y[..., :R].astype(np.float32)
    i1, i2 = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    a, b = f[..., i1], f[..., i2]
    y[..., i1] = (a * c - b * s).astype(np.float16)             # numpy rounds each float32 operation
    y[..., i2] = (b * c + a * s).astype(np.float16)
    return y


def kv_values(words, scales, bits, D):
    """float64 [groups, D] that cached groups stand for: (u - z) s, not rounded."""
    if bits == 16:
        return np.ascontiguousarray(words).view(np.float16).astype(np.float64).reshape(-1, D)
    u = kv_unpack(words, bits, D).astype(np.float64) - (1 << (bits - 1))
    return u * np.asarray(scales).view(np.float16).astype(np.float64).reshape(-1, 1)


def attention(q, k, v, pos, scale, causal=True, window=0):
    """One sequence: q float64 [n, heads, D], k, v [L, KV heads, D], pos [n] -> (out [n, heads, D], lse [n, heads],
    spread [n, heads, D] = sum w |v| / sum w, total [n, heads] = sum exp(s - max)). Rows that see nothing: 0 and -inf."""
    n, H, D = q.shape
    L, KH, _ = k.shape
    out, spread = np.zeros((n, H, D)), np.zeros((n, H, D))
    lse, total = np.full((n, H), -np.inf), np.ones((n, H))
    t = np.arange(L)
    for i in range(n):
        seen = np.ones(L, bool) if not causal else t <= pos[i]
        if window:
            seen &= t > pos[i] - window
        if not seen.any():
            continue
        for h in range(H):
            kh = h // (H // KH)
            x = (k[seen, kh] @ q[i, h]) * scale
            w = np.exp(x - x.max())
            out[i, h] = w @ v[seen, kh] / w.sum()
            spread[i, h] = w @ np.abs(v[seen, kh]) / w.sum()
            lse[i, h] = x.max() + np.log(w.sum())
            total[i, h] = w.sum()
    return out, lse, spread, total
