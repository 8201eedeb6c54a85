"""The example that runs quantised projections, rotary append, paged attention, fork and compaction together, against the
same block in 64 bits."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import paged_decode
    return paged_decode


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_paged_decode_example(example, bits):
    import torch
    exq = example.exq
    H, heads, kvh, D, prompt, forks, steps = 256, 4, 2, 64, 75, 3, 6
    block, (xp, xs), (yp, ys), ms, moved = example.run(hidden=H, heads=heads, kv_heads=kvh, D=D, bits=bits, page_size=16,
                                                       prompt=prompt, chunk=40, forks=forks, steps=steps)
    assert ms > 0 and moved > 0
    held = np.flatnonzero(block.refs)
    assert held.size == held[-1] + 1 and block.refs.max() == forks - 1      # compact; the prompt's whole pages are shared

    def dense(w):
        W = torch.empty(w.K, w.N, dtype=torch.float16, device="cuda")
        exq.exq_dequant(w, W)
        return W.double()

    Wq, Wk, Wv = (dense(w) for w in block.qkv)
    Wo = dense(block.o)
    freqs, _ = exq.exq_rope_freqs(D)

    def turn(x):  # [T, h, D], positions 0 .. T - 1, pairs (i, i + D / 2)
        a = torch.arange(x.shape[0], device="cuda", dtype=torch.float64)[:, None, None] * torch.from_numpy(freqs).cuda()
        u, w = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([u * a.cos() - w * a.sin(), u * a.sin() + w * a.cos()], -1)

    for f in range(forks):
        n = steps if f > 0 else steps // 2
        x = torch.cat([xp, xs[:n, f]]).double()
        got = torch.cat([yp, ys[:n, f]]).double()
        L = x.shape[0]
        q, k, v = turn((x @ Wq).view(L, heads, D)), turn((x @ Wk).view(L, kvh, D)), (x @ Wv).view(L, kvh, D)
        # fp16 after the projection (half a step, 2^-11) and after the turn (the pair's length bounds the first one's share),
        # fp32 sums of 256 terms far below that; then at most one step of the cache's codes
        pair = lambda t: torch.hypot(t[..., :D // 2], t[..., D // 2:]).repeat(1, 1, 2)  # noqa: E731
        step = lambda t: 0.0 if bits == 16 else t.abs().amax(-1, keepdim=True) * 1.01 / (2 ** (bits - 1) - 1)  # noqa: E731
        eq, ek, ev = pair(q) * 2.0 ** -9.9, pair(k) * 2.0 ** -9.9 + step(k), v.abs() * 2.0 ** -10.9 + step(v)
        q, k, v, eq, ek, ev = (t.repeat_interleave(heads // t.shape[1], 1) for t in (q, k, v, eq, ek, ev))
        dot = lambda a, b: torch.einsum("ihd,jhd->hij", a, b) * D ** -0.5  # noqa: E731
        mask = torch.ones(L, L, dtype=torch.bool, device="cuda").tril()
        p = dot(q, k).masked_fill(~mask, -torch.inf).softmax(-1)
        o = torch.einsum("hij,jhd->ihd", p, v)
        # a logit is off by ds at most: each weight by a factor within exp(2 max ds)
        ds = (dot(q.abs() + eq, ek) + dot(eq, k.abs())).masked_fill(~mask, 0).amax(-1)     # [heads, L]
        wide = torch.expm1(2 * ds + 2.0 ** -9).T[..., None]                                # weights as fp16: 2^-10 more
        spread = torch.einsum("hij,jhd->ihd", p, v.abs()) + o.abs()
        eo = wide * spread + torch.einsum("hij,jhd->ihd", p, ev) * (1 + wide) + o.abs() * 2.0 ** -10
        y = o.reshape(L, -1) @ Wo
        ey = eo.reshape(L, -1) @ Wo.abs() + y.abs() * 2.0 ** -10 + 1e-4
        assert bool(((got - y).abs() <= ey).all()), f
        if bits >= 8:  # and far below that bound as a whole
            assert float((got - y).norm() / y.norm()) < (2e-2 if bits == 8 else 4e-3)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
