"""GPU parity of exq_rope against the oracle, bit for bit, and of its gradient."""
from __future__ import annotations

import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch

    import __graft_entry__
    __graft_entry__.build()
    import quantized_weight_exq_gb300 as exq
    torch.cuda.set_device(0)
    return exq, torch


def _bits(a):
    return np.ascontiguousarray(a).view(np.uint16)


# (tokens, heads, D, R): whole and part of the head, pair chunks aligned and not, odd counts
SHAPES = [(1, 64, 128, 128), (1, 1, 8, 2), (37, 5, 64, 64), (300, 8, 128, 64), (7, 3, 256, 256), (19, 2, 128, 20),
          (5, 9, 80, 72), (3, 4, 512, 512), (11, 1, 24, 16), (700, 2, 128, 128), (6, 3, 512, 66)]


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("T,H,D,R", SHAPES)
def test_rope_bit_exact(env, T, H, D, R, layout):
    exq, torch = env
    rng = np.random.default_rng(T * 1000 + D + layout)
    x = (rng.standard_normal((T, H, D)) * 4).astype(np.float16)
    pos = np.concatenate([[0, -1, 2 ** 31 - 1, -2 ** 31, 131071][:T], rng.integers(-5, 1 << 20, max(0, T - 5))]).astype(np.int32)
    gain = 1.0 if layout else 1.2079441541679836
    f, _ = exq.exq_rope_freqs(R)
    steps = exq.exq_rope_steps(f)
    rope = exq.Rope(torch.from_numpy(steps.view(np.int64)).cuda(), R, layout, gain)
    xd, pd = torch.from_numpy(x).cuda(), torch.from_numpy(pos).cuda()
    for grad in (False, True):
        y = exq.exq_rope(xd, pd, rope, grad=grad)
        torch.cuda.synchronize()
        assert np.array_equal(_bits(y.cpu().numpy()), _bits(O.rope(x, steps, pos, R, bool(layout), gain, grad))), grad


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("R", [128, 36])
def test_rope_strides_and_in_place(env, R, layout):
    exq, torch = env
    rng = np.random.default_rng(R)
    T, H, D = 45, 6, 128
    whole = torch.from_numpy(rng.standard_normal((T, H + 5, D)).astype(np.float16)).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 977
    rope = exq.rope_table(R, layout)
    x = whole[:, 2:2 + H]                                     # strided rows
    ref = exq.exq_rope(x.contiguous(), pos, rope)
    out = torch.zeros(H, T, D, dtype=torch.float16, device="cuda").transpose(0, 1)   # heads outermost
    exq.exq_rope(x, pos, rope, out=out)
    before = whole.clone()
    exq.exq_rope(x, pos, rope, out=x)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(x, ref)
    assert torch.equal(whole[:, :2], before[:, :2]) and torch.equal(whole[:, 2 + H:], before[:, 2 + H:])


def test_rope_gradient_against_differences(env):
    # <g, rope(x + e) - rope(x - e)> = <2 e, grad(g)> up to fp16 roundings: each result and each gradient entry is off by
    # at most half a step (2^-11 of it) plus fp32 roundings far below
    exq, torch = env
    rng = np.random.default_rng(5)
    T, H, D, R = 33, 4, 64, 48
    for layout in (0, 1):
        rope = exq.rope_table(R, layout, scaling=exq.ROPE_SCALE_YARN, factor=4.0, orig_ctx=4096.0)
        assert rope.gain != 1.0
        pos = torch.arange(T, dtype=torch.int32, device="cuda") + 50000
        x = rng.integers(-8, 9, (T, H, D)).astype(np.float16)
        e = rng.integers(-8, 9, (T, H, D)).astype(np.float16)
        g = rng.integers(-8, 9, (T, H, D)).astype(np.float16)
        a = exq.exq_rope(torch.from_numpy(x + e).cuda(), pos, rope).double().cpu().numpy()
        b = exq.exq_rope(torch.from_numpy(x - e).cuda(), pos, rope).double().cpu().numpy()
        d = exq.exq_rope(torch.from_numpy(g).cuda(), pos, rope, grad=True).double().cpu().numpy()
        gd, ed = g.astype(np.float64), e.astype(np.float64)
        off = (np.abs(gd) * (np.abs(a) + np.abs(b))).sum((1, 2)) + (2 * np.abs(ed) * np.abs(d)).sum((1, 2))
        lhs, rhs = (gd * (a - b)).sum((1, 2)), (2 * ed * d).sum((1, 2))
        assert np.all(np.abs(lhs - rhs) <= off * (2.0 ** -11 + 2.0 ** -20)), layout


def test_rope_empty_stream_and_refusals(env):
    exq, torch = env
    rope = exq.rope_table(64)
    x = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    assert exq.exq_rope(x, torch.empty(0, dtype=torch.int32, device="cuda"), rope).shape == (0, 4, 64)
    x = torch.randn(9, 4, 64, device="cuda").half()
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    ref = exq.exq_rope(x, pos, rope)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = exq.exq_rope(x, pos, rope)
    s.synchronize()
    assert torch.equal(ref, other)
    for kw in (dict(x=x.float()), dict(pos=pos.long()), dict(pos=pos[:8]), dict(x=x[..., ::2]),
               dict(out=torch.empty(9, 4, 32, dtype=torch.float16, device="cuda"))):
        with pytest.raises(exq.ExqError):
            exq.exq_rope(**{**dict(x=x, pos=pos, rope=rope), **kw})
