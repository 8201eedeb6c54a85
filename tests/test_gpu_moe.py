"""The expert layer for a few tokens against the 64-bit oracle: routing, products, unused and repeated places."""
from __future__ import annotations

import numpy as np
import pytest

import oracle as O
from helpers import ulp16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch

    import __graft_entry__
    __graft_entry__.build()
    import quantized_weight_exq_gb300 as exq
    torch.cuda.set_device(0)
    return exq, torch


class Experts:
    """Random experts: the library's and the oracle's."""

    def __init__(self, exq, torch, fmt, E, D, I, seed, with_factors=True):
        rng = self.rng = np.random.default_rng(seed)
        self.E, self.D, self.I, self.fmt = E, D, I, fmt
        self.parts, self.values = [], []
        for rows, K in ((I, D), (I, D), (D, I)):
            codes = rng.integers(0, 16, (E, rows, K), dtype=np.uint8)
            blocks = K // O.FP4_BLOCK[fmt]
            if fmt == 1:
                scales = rng.integers(0x28, 0x38, (E, rows, blocks), dtype=np.uint8)
                factors = ((0.5 + rng.random(E)) * 2 / np.sqrt(K)).astype(np.float32) if with_factors else None
            else:
                mid = 127 - int(np.log2(np.sqrt(K))) - 2
                scales, factors = rng.integers(mid, mid + 3, (E, rows, blocks), dtype=np.uint8), None
            packed = [exq.exq_pack_fp4(c, s, fmt) for c, s in zip(codes, scales)]
            self.parts.append(exq.Fp4Experts(torch.from_numpy(np.stack([p for p, _ in packed])).cuda(),
                                             torch.from_numpy(np.stack([t for _, t in packed])).cuda(), fmt,
                                             None if factors is None else torch.from_numpy(factors).cuda()))
            self.values.append(lambda e, c=codes, s=scales, f=factors: O.fp4_values(c[e], s[e], fmt, 1.0 if f is None else f[e]))
        self.x = rng.standard_normal((16, D)).astype(np.float16)
        self.router = (rng.standard_normal((E, D)) * 1.5 / np.sqrt(D)).astype(np.float16)

    def reference(self, x, ids, weights, act=0):
        """(y, the size of what its sums add up: a bound's measure)"""
        x = np.asarray(x, np.float64)
        y, size = np.zeros_like(x), np.zeros_like(x)
        g, u, d = self.values
        for t in range(x.shape[0]):
            for e, w in zip(ids[t], weights[t]):
                if e < 0:
                    continue
                gv, uv = g(e) @ x[t], u(e) @ x[t]
                h = O.moe_activate(gv, act) * uv
                y[t] += float(w) * (d(e) @ h)
                # how far h may be off: the sums of gate and up (|act'| <= 1.13), 22 bits of h itself
                eg, eu = (np.abs(m(e)) @ np.abs(x[t]) * ((self.D / 16 + 170) * 2.0 ** -23) for m in (g, u))
                off = 1.13 * eg * (np.abs(uv) + eu) + np.abs(O.moe_activate(gv, act)) * eu + np.abs(h) * 2.0 ** -20
                size[t] += abs(float(w)) * (np.abs(d(e)) @ (off + (self.I / 16 + 170) * 2.0 ** -23 * np.abs(h)))
        return y, size

    def check(self, y, x, ids, weights, act=0):
        ref, size = self.reference(x, ids, weights, act)
        y = y.cpu().numpy().astype(np.float64)
        tol = 0.5 * ulp16(ref) * (1 + 2.0 ** -8) + size + 2.0 ** -22 * np.abs(ref) + 2.0 ** -24
        # 65520 and more is infinite in fp16; what lies within tol of it may be either
        over = np.abs(ref) - tol >= 65520
        assert (y[over] == np.sign(ref[over]) * np.inf).all()
        edge = (np.abs(ref) + tol >= 65520) & ~over
        assert np.isfinite(y[~over & ~edge]).all()
        with np.errstate(invalid="ignore"):
            err = np.where(over | edge, 0, np.abs(y - ref))
        assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size} off, by {np.max(err / tol):.3g} times what is allowed"


CASES = [  # format, experts, D, I, top_k, tokens, renorm
    (1, 8, 256, 128, 2, 1, True), (2, 8, 256, 128, 2, 1, True), (1, 4, 32, 32, 1, 3, False), (2, 6, 96, 160, 6, 16, False),
    (1, 16, 544, 288, 4, 5, True), (2, 60, 128, 96, 8, 9, True), (1, 128, 288, 64, 8, 16, False), (2, 3, 1056, 416, 2, 8, True),
    (1, 40, 2048, 544, 6, 16, True), (2, 512, 64, 32, 16, 7, True), (1, 1, 64, 96, 1, 2, True),
]


@pytest.mark.parametrize("fmt,E,D,I,k,T,renorm", CASES)
def test_layer(env, fmt, E, D, I, k, T, renorm):
    exq, torch = env
    ex = Experts(exq, torch, fmt, E, D, I, E + D + T)
    layer = exq.MoeLayer(*ex.parts, top_k=k, router=torch.from_numpy(ex.router).cuda(), renorm=renorm)
    x = torch.from_numpy(ex.x[:T]).cuda()
    out = torch.full((T, D), float("nan"), dtype=torch.float16, device="cuda")
    ws = torch.zeros(exq.exq_moe_workspace_size(layer, T), dtype=torch.uint8, device="cuda")
    y, ids, weights = exq.exq_moe(layer, x, out=out, workspace=ws)
    assert y is out and exq.exq_get_last_device_error() == exq.EXQ_OK
    assert not ws[:exq.FP4_COUNTER_BYTES].any()
    logits = ex.x[:T].astype(np.float64) @ ex.router.astype(np.float64).T
    rids, rw = O.moe_route(logits, k, renorm)
    # logits are off by at most D 2^-24 of their terms' magnitudes: experts nearer than that may change places
    near = D * 2.0 ** -23 * (np.abs(ex.x[:T].astype(np.float64)) @ np.abs(ex.router.astype(np.float64)).T).max()
    got = ids.cpu().numpy()
    for t in range(T):
        assert len(set(got[t])) == k
        assert np.abs(logits[t, got[t]] - logits[t, rids[t]]).max() <= near
    w = weights.cpu().numpy()
    rw = np.take_along_axis(np.exp(logits - logits.max(-1, keepdims=True)), got, -1)
    rw /= rw.sum(-1, keepdims=True) if renorm else np.exp(logits - logits.max(-1, keepdims=True)).sum(-1, keepdims=True)
    np.testing.assert_allclose(w, rw, rtol=4 * near + 2.0 ** -20)
    ex.check(y, ex.x[:T], got, w)
    y2, ids2, w2 = exq.exq_moe(layer, x)
    assert torch.equal(y, y2) and torch.equal(ids, ids2) and torch.equal(weights, w2)


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("act", [0, 1])
def test_given_places(env, fmt, act):
    # unused places, a token without experts, one that names an expert twice, all tokens on one expert, weights of either sign
    exq, torch = env
    ex = Experts(exq, torch, fmt, 10, 288, 160, 3 + fmt, with_factors=act == 0)
    layer = exq.MoeLayer(*ex.parts, top_k=3, act=act)
    for ids in ([[-1, -1, -1], [2, -1, 9], [4, 4, 4], [0, 4, 0]], [[5, -1, -1]] * 16, [[-1, 7, -1]], [[-1, -1, -1]] * 9,
                [[0, 1, 2], [3, 4, 5], [6, 7, 8], [9, 0, 1]] * 4):
        T = len(ids)
        ids = np.array(ids, np.int32)
        weights = ex.rng.standard_normal((T, 3)).astype(np.float32)
        out = torch.full((T, 288), float("nan"), dtype=torch.float16, device="cuda")
        y, i2, w2 = exq.exq_moe(layer, torch.from_numpy(ex.x[:T]).cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(weights).cuda(), out=out)
        assert exq.exq_get_last_device_error() == exq.EXQ_OK
        np.testing.assert_array_equal(i2.cpu().numpy(), ids)   # read only
        np.testing.assert_array_equal(w2.cpu().numpy(), weights)
        ex.check(y, ex.x[:T], ids, weights, act)
        for t in range(T):
            if (ids[t] < 0).all():
                assert not y[t].any()


def test_bad_places_are_reported_and_skipped(env):
    exq, torch = env
    ex = Experts(exq, torch, 1, 5, 64, 64, 1)
    layer = exq.MoeLayer(*ex.parts, top_k=2)
    ids = np.array([[0, 5], [-2, 3], [1, 2 ** 31 - 1], [-(2 ** 31), -1]], np.int32)
    weights = np.full((4, 2), 0.5, np.float32)
    y, _, _ = exq.exq_moe(layer, torch.from_numpy(ex.x[:4]).cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(weights).cuda())
    assert exq.exq_get_last_device_error() == exq.EXQ_ERR_INVALID_ARG
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    ex.check(y, ex.x[:4], np.where((ids >= 0) & (ids < 5), ids, -1), weights)


def test_routing_of_ties_and_what_is_not_finite(env):
    exq, torch = env
    E, D, k = 40, 64, 5
    ex = Experts(exq, torch, 1, E, D, 32, 2)
    router = np.zeros((E, D), np.float16)
    router[3, 0], router[17, 0], router[39, 0], router[30, 0] = 1, 1, 1, -1
    router[5, 1], router[6, 2] = np.nan, np.inf
    x = np.zeros((4, D), np.float16)
    x[0, 0], x[1, 3], x[2, 2], x[3, 0] = 2, 1, 1, np.nan
    layer = exq.MoeLayer(*ex.parts, top_k=k, router=torch.from_numpy(router).cuda())
    y, ids, w = exq.exq_moe(layer, torch.from_numpy(x).cuda())
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    # token 0: NaN for experts 5 (0 * NaN) and 6 (0 * inf), ties at 2 and at 0
    assert ids[0].tolist() == [3, 17, 39, 0, 1] and ids[1].tolist() == [0, 1, 2, 3, 4]
    np.testing.assert_allclose(w[0], np.exp([0, 0, 0, -2, -2]) / np.exp([0, 0, 0, -2, -2]).sum(), rtol=1e-6)
    np.testing.assert_allclose(w[1], 0.2, rtol=1e-6)
    assert ids[2].tolist() == [6, 0, 1, 2, 3] and np.isnan(w[2, 0])     # inf - inf
    assert ids[3].tolist() == [0, 1, 2, 3, 4] and np.isnan(w[3]).all()  # nothing but NaN: the first places
    assert np.isfinite(y[:2].float().cpu().numpy()).all()
    # the NaNs of tokens 2 and 3 stay with them
    z, _, _ = exq.exq_moe(exq.MoeLayer(*ex.parts, top_k=k), torch.from_numpy(x[:2]).cuda(), torch.from_numpy(ids[:2]).cuda(), torch.from_numpy(w[:2]).cuda())
    ex.check(y[:2], x[:2], ids[:2], w[:2])
    ex.check(z, x[:2], ids[:2], w[:2])


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("part", [0, 1, 2])
def test_a_spoilt_expert_reaches_its_tokens_only(env, fmt, part):
    exq, torch = env
    ex = Experts(exq, torch, fmt, 6, 96, 160, 5)
    layer = exq.MoeLayer(*ex.parts, top_k=2)
    ids = np.array([[0, 1], [2, 3], [4, 5], [3, 0]], np.int32)
    weights = np.full((4, 2), 0.5, np.float32)
    args = [torch.from_numpy(a).cuda() for a in (ex.x[:4], ids, weights)]
    want = exq.exq_moe(layer, *args)[0]
    ex.parts[part].scales[3].fill_(0x7F if fmt == 1 else 0xFF)
    got = exq.exq_moe(layer, *args)[0]
    assert torch.isnan(got[[1, 3]]).all()
    assert torch.equal(got[[0, 2]], want[[0, 2]])


def test_graph_of_routing_and_experts(env):
    # replayed on other tokens, which choose other experts; a second graph with a workspace of its own beside it
    exq, torch = env
    ex = Experts(exq, torch, 1, 24, 256, 160, 9)
    layer = exq.MoeLayer(*ex.parts, top_k=4, router=torch.from_numpy(ex.router).cuda())
    T = 6
    x = torch.from_numpy(ex.x[:T]).cuda()
    made = []
    for _ in range(2):
        ws = torch.zeros(exq.exq_moe_workspace_size(layer, T), dtype=torch.uint8, device="cuda")
        out = [torch.empty(T, 256, dtype=torch.float16, device="cuda"), torch.empty(T, 4, dtype=torch.int32, device="cuda"),
               torch.empty(T, 4, dtype=torch.float32, device="cuda")]
        exq.exq_moe(layer, x, out[1], out[2], out[0], ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            exq.exq_moe(layer, x, out[1], out[2], out[0], ws)
        made.append((graph, out, ws))
    for first in (4, 10):
        x.copy_(torch.from_numpy(ex.x[first:first + T]))
        for graph, out, _ in made:
            out[0].fill_(float("nan"))
        streams = [torch.cuda.Stream() for _ in made]
        for (graph, _, _), s in zip(made, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        want = exq.exq_moe(layer, x)
        for _, out, _ in made:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
        ex.check(want[0], ex.x[first:first + T], want[1].cpu().numpy(), want[2].cpu().numpy())
    with pytest.raises(exq.ExqError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            exq.exq_moe(layer, x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = exq.exq_moe(layer, x, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(z, want))


def test_refusals(env):
    exq, torch = env
    ex = Experts(exq, torch, 1, 4, 64, 32, 9)
    g, u, d = ex.parts
    layer = exq.MoeLayer(g, u, d, top_k=2)
    x = torch.from_numpy(ex.x[:2]).cuda()
    ids, w = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, 2, device="cuda")
    router = torch.zeros(4, 64, dtype=torch.float16, device="cuda")
    for call in (lambda: exq.exq_moe(layer, x), lambda: exq.exq_moe(layer, x, ids), lambda: exq.exq_moe(layer, x, ids.long(), w),
                 lambda: exq.exq_moe(layer, x, ids, w.half()), lambda: exq.exq_moe(layer, x, ids[:1], w), lambda: exq.exq_moe(layer, x.float(), ids, w),
                 lambda: exq.exq_moe(layer, x.repeat(9, 1), ids.repeat(9, 1), w.repeat(9, 1)), lambda: exq.exq_moe(layer, x[:0], ids[:0], w[:0]),
                 lambda: exq.exq_moe(layer, x, ids, w, out=x[:1]), lambda: exq.exq_moe(layer, x, ids.cpu(), w),
                 lambda: exq.exq_moe(layer, x, ids, w, workspace=torch.zeros(1 << 17, dtype=torch.uint8, device="cuda")),
                 lambda: exq.MoeLayer(g, u, d, top_k=2, router=router[:3]), lambda: exq.MoeLayer(g, u, d, top_k=2, router=router.float()),
                 lambda: exq.exq_moe(exq.MoeLayer(g, d, u, top_k=2, router=router), x), lambda: exq.exq_moe(exq.MoeLayer(g, u, d, top_k=5, router=router), x),
                 lambda: exq.Fp4Experts(g.codes, g.scales[:3], 1), lambda: exq.Fp4Experts(g.codes, g.scales, 1, w[0])):
        with pytest.raises(exq.ExqError):
            call()
    assert exq.exq_get_last_device_error() == exq.EXQ_OK


def test_waits_run_out_then_recover(env):
    exq, torch = env
    ex = Experts(exq, torch, 2, 8, 512, 256, 11)
    layer = exq.MoeLayer(*ex.parts, top_k=2, router=torch.from_numpy(ex.router).cuda())
    x = torch.from_numpy(ex.x[:3]).cuda()
    ws = torch.zeros(exq.exq_moe_workspace_size(layer, 3), dtype=torch.uint8, device="cuda")
    want = exq.exq_moe(layer, x, workspace=ws)[0]
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    exq.exq_testing_starve(64)
    try:
        exq.exq_moe(layer, x, workspace=ws)
        assert exq.exq_get_last_device_error() == exq.EXQ_ERR_TIMEOUT
    finally:
        exq.exq_testing_starve(0)
    ws[:exq.FP4_COUNTER_BYTES].zero_()
    assert torch.equal(exq.exq_moe(layer, x, workspace=ws)[0], want)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("T", [1, 2, 13])
def test_steps_of_a_decode_loop(env, fmt, T):
    # each call reads what the one before it wrote, weights among it, and begins while that one ends: the bits are those of
    # calls with a synchronise between them, from the host and from a graph
    exq, torch = env
    D = 512
    ex = Experts(exq, torch, fmt, 12, D, 288, 21)
    layer = exq.MoeLayer(*ex.parts, top_k=3, router=torch.from_numpy(ex.router).cuda())
    x0 = torch.from_numpy(ex.x[:T]).cuda()
    gen = torch.Generator(device="cuda").manual_seed(4)
    dense = [torch.randn(D, D, generator=gen, device="cuda").half() / 16 for _ in range(6)]
    w = exq.exq_fp4_quantize(dense[0], fmt)
    ws = torch.zeros(max(exq.exq_moe_workspace_size(layer, T), exq.exq_fp4_gemv_workspace_size(w, T)), dtype=torch.uint8, device="cuda")
    ys = [torch.empty(T, D, dtype=torch.float16, device="cuda") for _ in range(3 * len(dense))]
    ids, weights = torch.empty(T, 3, dtype=torch.int32, device="cuda"), torch.empty(T, 3, dtype=torch.float32, device="cuda")

    def steps(between):
        x = x0
        for i, d in enumerate(dense):
            a, b, c = ys[3 * i:3 * i + 3]
            exq.exq_fp4_quantize(d, fmt, out=w), between()
            exq.exq_fp4_gemv(w, x, out=a, workspace=ws), between()
            exq.exq_moe(layer, a, ids, weights, out=b, workspace=ws), between()
            exq.exq_fp4_quantize(b, fmt, out=rows), between()
            exq.exq_fp4_gemm(rows, w, out=c), between()
            x = torch.add(x0, c, alpha=2.0 ** -10, out=xs[i])

    xs = torch.empty(len(dense), T, D, dtype=torch.float16, device="cuda")
    rows = exq.exq_fp4_quantize(x0, fmt)
    steps(torch.cuda.synchronize)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    want = [y.view(torch.int16).clone() for y in ys]
    assert all(torch.isfinite(y).all() and y.any() for y in ys)
    for _ in range(20):
        for y in ys:
            y.fill_(float("nan"))
        steps(lambda: None)
        assert all(torch.equal(y.view(torch.int16), v) for y, v in zip(ys, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps(lambda: None)
    for _ in range(20):
        for y in ys:
            y.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(y.view(torch.int16), v) for y, v in zip(ys, want))
    assert not ws[:exq.FP4_COUNTER_BYTES].any()


@pytest.mark.parametrize("fmt", [1, 2])
def test_threads_on_one_stream(env, fmt):
    # host threads whose calls of several launches share a stream's default workspace: the bits are those of calls one by one
    import threading
    exq, torch = env
    ex = Experts(exq, torch, fmt, 12, 512, 288, 23 + fmt)
    layer = exq.MoeLayer(*ex.parts, top_k=3, router=torch.from_numpy(ex.router).cuda())
    gen = torch.Generator(device="cuda").manual_seed(fmt)
    w = exq.exq_fp4_quantize(torch.randn(2056, 1024, generator=gen, device="cuda").half() / 16, fmt)
    xs = [torch.randn(m, 1024, generator=gen, device="cuda").half() for m in (16, 9, 16, 3)]
    ts = [torch.randn(t, 512, generator=gen, device="cuda").half() for t in (16, 5, 1, 13)]
    jobs = [lambda x=x: [exq.exq_fp4_gemv(w, x)] for x in xs] + [lambda x=x: exq.exq_moe(layer, x) for x in ts]
    exq.exq._fp4_ws.clear()  # so that it grows again while the threads run
    torch.cuda.synchronize()
    want = [[t.clone() for t in job()] for job in jobs]
    torch.cuda.synchronize()
    exq.exq._fp4_ws.clear()
    got, errors = [[] for _ in jobs], []

    def work(i):
        try:
            torch.cuda.set_device(0)
            for _ in range(50):
                got[i].append(jobs[i]())
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and exq.exq_get_last_device_error() == exq.EXQ_OK
    for results, ref in zip(got, want):
        assert len(results) == 50
        for r in results:
            assert all(torch.equal(a, b) for a, b in zip(r, ref))


def _layer_of(exq, torch, fmt, parts, top_k, act=0):
    """A layer from (codes [E, rows, K], scale bytes, factors or None) of gate, up and down, and their values in 64 bits."""
    made, values = [], []
    for codes, scales, factors in parts:
        codes, scales = codes.astype(np.uint8), scales.astype(np.uint8)
        packed = [exq.exq_pack_fp4(c, s, fmt) for c, s in zip(codes, scales)]
        made.append(exq.Fp4Experts(torch.from_numpy(np.stack([p for p, _ in packed])).cuda(), torch.from_numpy(np.stack([t for _, t in packed])).cuda(),
                                   fmt, None if factors is None else torch.from_numpy(np.float32(factors)).cuda()))
        values.append(np.stack([O.fp4_values(c, s, fmt, 1.0 if factors is None else factors[e]) for e, (c, s) in enumerate(zip(codes, scales))]))
    return exq.MoeLayer(*made, top_k=top_k, act=act), values


def _power(fmt, e):
    """(a scale byte and a factor that are 2^e together, the factor None for E8M0)"""
    return (0x38, 2.0 ** e) if fmt == 1 else (127 + e, None)


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("T", [1, 2, 12])
def test_h_up_to_the_largest_numbers(env, fmt, T):
    # h up to 1.92 * 2^127, brought back by down's scales and the tokens' weights
    exq, torch = env
    rng = np.random.default_rng(T + fmt)
    D, I, block = 32, 96, O.FP4_BLOCK[fmt]
    gate, up = np.zeros((1, I, D)), np.zeros((1, I, D))
    gate[0, :, 0], up[0, :, 0] = 3, rng.integers(1, 3, I)      # 1.5; 0.5 or 1
    up[0, 5, 0] = 2
    up[0, :, 0] += 8 * rng.integers(0, 2, I)
    down = rng.integers(0, 16, (1, D, I))
    (sg, fg), (su, fu), (sd, fd) = (_power(fmt, e) for e in (63, 63, -100))
    parts = [(c, np.full((1, c.shape[1], c.shape[2] // block), s), None if f is None else [f])
             for c, s, f in ((gate, sg, fg), (up, su, fu), (down, sd, fd))]
    layer, (gv, uv, dv) = _layer_of(exq, torch, fmt, parts, 1)
    x = np.zeros((T, D), np.float16)
    x[:, 0] = np.resize([1.29, 1.6, 1.25, 1.15], T)
    weights = np.full((T, 1), 2.0 ** -24, np.float32)
    y, _, _ = exq.exq_moe(layer, torch.from_numpy(x).cuda(), torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.from_numpy(weights).cuda())
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    for t in range(T):
        h = (gv[0] @ x[t].astype(np.float64)) * (uv[0] @ x[t].astype(np.float64))  # (SiLU of what is so large is itself)
        assert 2.0 ** 126 < np.abs(h).max() < 2.0 ** 128 and (t % 4 == 3 or np.abs(h).max() > 2.0 ** 127)
        ref, size = dv[0] @ h * 2.0 ** -24, np.abs(dv[0]) @ np.abs(h) * 2.0 ** -24
        assert 1 < np.abs(ref).max() < 65504
        # gate's and up's sums have one term: h is off by its own rounding, 2^-24, and by 2^-23 of its block's largest (at most
        # twice itself); then the sums' roundings and the result's
        tol = 0.5 * ulp16(ref) * (1 + 2.0 ** -8) + ((I / 16 + 170) * 2.0 ** -23 + 2.0 ** -24 + 2.0 ** -22) * size
        assert (np.abs(y[t].cpu().numpy().astype(np.float64) - ref) <= tol).all()


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("T", [1, 3])
def test_h_of_mixed_sizes(env, fmt, T):
    # one channel of h far above the other blocks, which alone reach the result: each is held to 2^-23 of its block's largest,
    # with e4m3 scales plus 2^-40 of the token's
    exq, torch = env
    rng = np.random.default_rng(T + fmt)
    D, I, block = 32, 160, O.FP4_BLOCK[fmt]
    gate = rng.integers(1, 8, (1, I, D)) + 8 * rng.integers(0, 2, (1, I, D))
    up = rng.integers(1, 8, (1, I, D)) + 8 * rng.integers(0, 2, (1, I, D))
    down = rng.integers(0, 16, (1, D, I))
    gate[:, 0] &= 7
    up[:, 0] &= 7
    down[:, :, :block] = 0
    su = np.full((1, I, D // block), 0x28 if fmt == 1 else 120)  # 2^-2, 2^-7
    for j in range(block, I, block):                             # blocks of h from 2^-9 to 2^-16 down (e4m3: of normal scales), or 2^-60
        su[0, j:j + block] = 0x10 - 8 * (j // block % 2) if fmt == 1 else 120 - 15 * (j // block)
    sg = np.full_like(su, 0x38 if fmt == 1 else 127)
    su[0, 0], sg[0, 0] = (0x78, 0x78) if fmt == 1 else (150, 127)  # channel 0: 2^8 and 2^8, or 2^23
    sd = np.full((1, D, I // block), 0x38 if fmt == 1 else 127 + 20)
    f = [[1.0] if fmt == 1 else None] * 3
    layer, (gv, uv, dv) = _layer_of(exq, torch, fmt, list(zip((gate, up, down), (sg, su, sd), f)), 1)
    x = np.abs(rng.standard_normal((T, D))).astype(np.float16)
    w = np.ones((T, 1), np.float32)
    y, _, _ = exq.exq_moe(layer, torch.from_numpy(x).cuda(), torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.from_numpy(w).cuda())
    for t in range(T):
        xt = x[t].astype(np.float64)
        g, u = gv[0] @ xt, uv[0] @ xt
        h = O.moe_activate(g, 0) * u
        largest = np.repeat(np.abs(h).reshape(-1, block).max(1), block)
        assert np.abs(h).max() > 2.0 ** 16 * np.abs(h[block:]).max()
        eg, eu = (np.abs(m[0]) @ np.abs(xt) * ((D / 16 + 170) * 2.0 ** -23) for m in (gv, uv))
        off = 1.13 * eg * (np.abs(u) + eu) + np.abs(O.moe_activate(g, 0)) * eu + 2.0 ** -20 * np.abs(h) + 2.0 ** -23 * largest
        if fmt == 1:
            off += 2.0 ** -40 * np.abs(h).max()
        ref = dv[0] @ h
        tol = 0.5 * ulp16(ref) * (1 + 2.0 ** -8) + np.abs(dv[0]) @ (off + (I / 16 + 170) * 2.0 ** -23 * np.abs(h))
        assert (np.abs(y[t].cpu().numpy().astype(np.float64) - ref) <= tol).all()


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("T", [1, 4, 16])
def test_gelu_of_what_it_hardly_lets_through(env, fmt, T):
    # a token whose gate is -6 to -2 everywhere: the result is small, and as precise as another
    exq, torch = env
    rng = np.random.default_rng(T + fmt)
    E, D, I, block = 4, 32, 64, O.FP4_BLOCK[fmt]
    gate, up = np.zeros((E, I, D)), np.zeros((E, I, D))
    gate[:, :, 0] = 8 + np.array([4, 5, 6, 7])[:, None]          # -2, -3, -4, -6
    up[:, :, 0] = rng.integers(2, 8, (E, I))
    down = rng.integers(1, 8, (E, D, I))                         # of one sign: no sum cancels
    factors = 2.0 ** np.array([0, 4, 8, 28])                     # of down: results in fp16's range
    scale = lambda rows, K: np.full((E, rows, K // block), 0x38 if fmt == 1 else 127)  # noqa: E731
    parts = [(gate, scale(I, D), None), (up, scale(I, D), None), (down, scale(D, I), factors)]
    if fmt == 2:
        parts[2] = (down, scale(D, I) + np.int64(np.log2(factors))[:, None, None], None)
    layer, (gv, uv, dv) = _layer_of(exq, torch, fmt, parts, 1, act=1)
    for first in range(E if T == 1 else 1):
        ids = ((first + np.arange(T)) % E).astype(np.int32)[:, None]
        x = np.zeros((T, D), np.float16)
        x[:, 0] = 1
        y, _, _ = exq.exq_moe(layer, torch.from_numpy(x).cuda(), torch.from_numpy(ids).cuda(), torch.ones(T, 1, device="cuda"))
        for t in range(T):
            e = ids[t, 0]
            g, u = gv[e, :, 0], uv[e, :, 0]
            ref = dv[e] @ (g / (1 + np.exp(-2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3))) * u)
            # the exponent is 25 at most, off by four roundings of 2^-24 of itself (6e-6), its exponential by 31 * 2^-23 (4e-6): 2^-16
            tol = 0.5 * ulp16(ref) * (1 + 2.0 ** -8) + (2.0 ** -16 + (I / 16 + 170) * 2.0 ** -23) * np.abs(ref)
            assert (np.abs(y[t].cpu().numpy().astype(np.float64) - ref) <= tol).all(), (e, y[t], ref)
