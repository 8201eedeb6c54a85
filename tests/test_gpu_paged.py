"""GPU parity of the paged KV cache: the append and the page copies bit for bit, attention within derived bounds."""
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


def _np(t):
    return t.cpu().numpy()


class Case:
    """A cache of `layers` layers whose every slot holds junk (NaN scales or NaN values), the pages of some sequences,
    scattered, and the step's batch. fill() writes the sequences' tokens, through the oracle's codec."""

    def __init__(self, exq, torch, bits, D, page, kv_heads, lens, news, layers=1, layer=0, seed=0, spare=3):
        self.exq, self.torch, self.rng = exq, torch, np.random.default_rng(seed)
        self.bits, self.D, self.page, self.KH, self.layer = bits, D, page, kv_heads, layer
        self.lens, self.news = list(lens), list(news)
        need = [-(-n // page) for n in lens]
        n_pages, width = sum(need) + spare, max(max(need), 1)
        ids = self.rng.permutation(n_pages)[:sum(need)]
        self.table = np.full((len(lens), width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        shape = (layers, n_pages, kv_heads, page)
        W = D * bits // 32
        if bits == 16:
            self.words = [np.full((*shape, W), 0x7E007E00, np.uint32) for _ in range(2)]   # NaN pairs
            self.scales = [None, None]
        else:
            self.words = [self.rng.integers(0, 1 << 32, (*shape, W), dtype=np.uint32) for _ in range(2)]
            self.scales = [np.full(shape, 0x7E00, np.uint16) for _ in range(2)]            # NaN
        self.start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)

    def fill(self, lo=0):
        """Tokens lo[b] .. lens[b] of every sequence, and what they stand for: self.dense[b] = (k, v) float64."""
        self.dense = []
        for b, n in enumerate(self.lens):
            pair = []
            for i in range(2):
                x = (self.rng.standard_normal((n, self.KH, self.D)) * np.exp2(self.rng.integers(-3, 3, (n, self.KH, 1))))
                x = x.astype(np.float16)
                pair.append(self.put(b, i, x, np.arange(n)))
            self.dense.append(pair)
        return self

    def put(self, b, i, x, pos):
        """Writes x [n, KV heads, D] at positions pos of sequence b; returns the values the groups stand for."""
        n = len(pos)
        if n == 0:
            return np.zeros((0, self.KH, self.D))
        pages, slots = self.table[b, pos // self.page], pos % self.page
        if self.bits == 16:
            w = np.ascontiguousarray(x).view(np.uint32).reshape(n, self.KH, -1)
            self.words[i][self.layer, pages, :, slots] = w
            return x.astype(np.float64)
        u, s = O.kv_quantize(x.reshape(-1, self.D), self.bits)
        w = O.kv_pack(u, self.bits)
        self.words[i][self.layer, pages, :, slots] = w.reshape(n, self.KH, -1)
        self.scales[i][self.layer, pages, :, slots] = s.reshape(n, self.KH)
        return O.kv_values(w, s, self.bits, self.D).reshape(n, self.KH, self.D)

    def read(self, b, i):
        """What sequence b's cached tokens of K (i = 0) or V (1) stand for, from the pool as it is: float64 [n, KV heads, D]."""
        pos = np.arange(self.lens[b])
        at = self.layer, self.table[b, pos // self.page], slice(None), pos % self.page
        s = self.scales[i] if self.scales[i] is None else self.scales[i][at].reshape(-1)
        with np.errstate(all="ignore"):
            v = O.kv_values(self.words[i][at].reshape(-1, self.words[i].shape[-1]), s, self.bits, self.D)
        return v.reshape(-1, self.KH, self.D)

    def cache(self):
        t = self.torch
        words = [t.from_numpy(w.view(np.int32)).cuda() for w in self.words]
        scales = [None if s is None else t.from_numpy(s.view(np.float16)).cuda() for s in self.scales]
        return self.exq.KVCache(*words, *scales, self.bits)

    def batch(self, rows=None, **kw):
        t = self.torch
        d = dict(max_q_len=max(self.news), max_kv_len=max(self.lens), n_tokens=rows)
        return self.exq.KVBatch(t.from_numpy(self.start).cuda(), t.tensor(self.lens, dtype=t.int32).cuda(),
                                t.from_numpy(self.table).cuda(), **{**d, **kw})

    def same(self, cache):
        """The pool on the GPU is exactly this one."""
        got = [cache.k_codes, cache.v_codes]
        for g, w in zip(got, self.words):
            assert np.array_equal(_np(g).view(np.uint32), w)
        for g, s in zip([cache.k_scales, cache.v_scales], self.scales):
            assert s is None or np.array_equal(_np(g).view(np.uint16), s)


# ---------------------------------------------------------------- append

APPENDS = [  # bits, D, page, KV heads, query heads, lens, news, R, interleaved
    (4, 128, 16, 8, 64, [17], [1], 128, False),
    (6, 128, 32, 2, 4, [1, 40, 33, 64], [1, 1, 1, 1], 128, True),
    (8, 64, 64, 3, 6, [70, 3, 0, 129], [66, 2, 0, 5], 64, False),
    (16, 256, 256, 1, 8, [300, 257], [258, 1], 256, True),
    (4, 256, 16, 2, 2, [50], [50], 20, False),
    (6, 64, 128, 4, 4, [200, 1], [199, 1], 6, True),
    (16, 128, 16, 5, 5, [33], [3], 32, False),
    (8, 128, 64, 8, 8, [1200, 700], [1100, 650], 128, False),
    (6, 256, 16, 1, 3, [40], [9], 18, False),
]


@pytest.mark.parametrize("case", APPENDS, ids=[f"{c[0]}-{c[1]}-{c[2]}-{sum(c[6])}" for c in APPENDS])
def test_append_bit_exact(env, case):
    exq, torch = env
    bits, D, page, KH, H, lens, news, R, inter = case
    c = Case(exq, torch, bits, D, page, KH, lens, news, layers=2, layer=1, seed=D + bits)
    T = sum(news)
    rng = c.rng
    qkv = rng.standard_normal((T + 2, H + 2 * KH, D)).astype(np.float16)          # two rows of padding
    qkv[0, :, :5] = [0, -0.0, 60000.0, 2.0 ** -24, 1e-4]
    gpu = torch.from_numpy(qkv).cuda()
    cache = c.cache()
    steps = exq.exq_rope_steps(exq.exq_rope_freqs(R)[0])
    rope = exq.Rope(torch.from_numpy(steps.view(np.int64)).cuda(), R, int(inter), 1.0)
    q_out = torch.full((T + 2, H, D), 7.0, dtype=torch.float16, device="cuda")
    exq.exq_kv_append(cache, c.batch(rows=T + 2), gpu[:, H:H + KH], gpu[:, H + KH:], q=gpu[:, :H], rope=rope, q_out=q_out, layer=1)
    pos = np.concatenate([np.arange(L - n, L) for n, L in zip(news, lens)]).astype(np.int64)
    qr, kr = (O.rope(qkv[:T, a], steps, pos, R, inter) for a in (slice(0, H), slice(H, H + KH)))
    for b, (n, L) in enumerate(zip(news, lens)):
        rows = slice(c.start[b], c.start[b + 1])
        c.put(b, 0, kr[rows], np.arange(L - n, L))
        c.put(b, 1, qkv[rows, H + KH:], np.arange(L - n, L))
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    c.same(cache)
    assert np.array_equal(_np(q_out[:T]).view(np.uint16), qr.view(np.uint16))
    assert torch.all(q_out[T:] == 7.0)
    assert np.array_equal(_np(gpu).view(np.uint16), qkv.view(np.uint16))


@pytest.mark.parametrize("bits", [4, 6, 8, 16])
def test_append_without_rope_and_with_positions(env, bits):
    exq, torch = env
    D, KH = 64, 2
    c = Case(exq, torch, bits, D, 16, KH, [20, 5], [18, 5], seed=bits)
    k, v = (c.rng.standard_normal((23, KH, D)).astype(np.float16) for _ in range(2))
    cache = c.cache()
    assert exq.exq_kv_append(cache, c.batch(), torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()) is None
    for b, rows, pos in ((0, slice(0, 18), np.arange(2, 20)), (1, slice(18, 23), np.arange(5))):
        c.put(b, 0, k[rows], pos)
        c.put(b, 1, v[rows], pos)
    torch.cuda.synchronize()
    c.same(cache)
    # positions of the caller's own, and q turned in place
    steps = exq.exq_rope_steps(exq.exq_rope_freqs(D)[0])
    rope = exq.Rope(torch.from_numpy(steps.view(np.int64)).cuda(), D)
    pos = c.rng.integers(-100, 1 << 20, 23).astype(np.int32)
    q = c.rng.standard_normal((23, 4, D)).astype(np.float16)
    qd = torch.from_numpy(q).cuda()
    out = exq.exq_kv_append(cache, c.batch(), torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), q=qd, rope=rope,
                            pos=torch.from_numpy(pos).cuda(), q_out=qd)
    kr = O.rope(k, steps, pos, D)
    c.put(0, 0, kr[:18], np.arange(2, 20))
    c.put(1, 0, kr[18:], np.arange(5))
    torch.cuda.synchronize()
    assert out is qd and np.array_equal(_np(qd).view(np.uint16), O.rope(q, steps, pos, D).view(np.uint16))
    c.same(cache)


def test_append_reports_bad_pages_and_lengths(env):
    # every one of these is found by the kernel's own checks before an address is made of it
    exq, torch = env
    D, KH = 64, 2
    k = torch.randn(4, KH, D, device="cuda").half()

    def run(spoil, **bounds):
        c = Case(exq, torch, 4, D, 16, KH, [20, 18], [2, 2], seed=3)
        spoil(c)
        cache = c.cache()
        exq.exq_kv_append(cache, c.batch(**bounds), k, k)
        return exq.exq_get_last_device_error(), c, cache

    assert run(lambda c: None)[0] == exq.EXQ_OK
    for bad in (-1, -2 ** 31, 2 ** 31 - 1):
        err, c, cache = run(lambda c: c.table.__setitem__((slice(None), 1), bad))
        assert err == exq.EXQ_ERR_INVALID_ARG
        c.same(cache)                                            # nothing written
    assert run(lambda c: None, max_kv_len=19)[0] == exq.EXQ_ERR_INVALID_ARG
    assert run(lambda c: None, max_q_len=1)[0] == exq.EXQ_ERR_INVALID_ARG
    assert run(lambda c: setattr(c, "lens", [1, 20]), max_kv_len=20)[0] == exq.EXQ_ERR_INVALID_ARG    # fewer cached than new
    assert run(lambda c: c.start.__setitem__(slice(None), [1, 2, 4]))[0] == exq.EXQ_ERR_INVALID_ARG   # does not begin at 0
    assert exq.exq_get_last_device_error() == exq.EXQ_OK


# ---------------------------------------------------------------- attention

ATTN = [  # bits, D, page, KV heads, query heads, lens, news, causal, window
    (4, 128, 256, 2, 16, [500], [1], True, 0),
    (4, 128, 16, 1, 8, [1, 2, 15, 16, 17, 63, 64, 65, 0], [1, 1, 1, 1, 1, 1, 1, 1, 1], True, 0),
    (6, 128, 32, 2, 8, [700, 33], [1, 1], True, 0),
    (8, 128, 64, 1, 1, [1000, 129], [1, 1], True, 0),
    (16, 128, 64, 3, 3, [300, 77, 1], [1, 1, 1], True, 0),
    (4, 64, 32, 2, 10, [333, 40], [3, 1], True, 0),
    (6, 64, 16, 2, 8, [100, 257], [5, 5], True, 0),
    (8, 64, 256, 1, 4, [500], [7], True, 100),
    (16, 64, 16, 2, 4, [90, 31], [9, 31], True, 0),
    (4, 256, 64, 1, 4, [200, 65], [1, 2], True, 0),
    (6, 256, 16, 1, 2, [150], [3], True, 64),
    (8, 256, 128, 1, 8, [260], [1], False, 0),
    (16, 256, 32, 1, 6, [130, 20], [4, 20], True, 17),
    (4, 128, 64, 1, 8, [300], [130], True, 0),
    (8, 128, 16, 2, 4, [200, 90, 5], [200, 70, 5], True, 0),
    (6, 128, 64, 1, 5, [333], [111], True, 50),
    (16, 128, 128, 1, 2, [400, 129], [150, 129], True, 0),
    (16, 128, 16, 2, 2, [270], [270], True, 33),
    (4, 64, 16, 1, 4, [290], [290], True, 0),
    (16, 64, 64, 2, 16, [190, 64], [64, 64], False, 0),
    (8, 64, 32, 1, 3, [260], [97], True, 0),
    (6, 64, 64, 1, 8, [140], [60], True, 0),
    (4, 256, 32, 1, 4, [210], [80], True, 0),
    (16, 256, 64, 1, 2, [150, 70], [140, 70], True, 0),
    (8, 256, 16, 1, 8, [90], [33], True, 40),
    (6, 256, 64, 1, 3, [180], [129], True, 0),
    (4, 128, 16, 2, 8, [3, 10, 40], [8, 10, 20], True, 0),     # more new tokens than cached ones: rows that see nothing
    (16, 128, 16, 1, 4, [0, 2, 300], [70, 70, 70], True, 0),
]


def _bound(ref, spread, total, q, k, v, scale, n, D):
    """How far an output may be: the result's rounding and each weight's to fp16 (2^-11 relative), weights under fp16's
    normal range (2^-25 of the largest, with a factor 2 for V's scale brought to a power of two, times what a code can
    stand for), and the scores' fp32 sums (D products and the scale, 2^-24 each of their magnitudes), which move a weight by
    twice their error at most."""
    big = np.abs(q).sum(-1).max() * np.abs(k).max() * abs(scale)
    score = (D + 8) * 2.0 ** -24 * big
    tiny = 4 * n * 2.0 ** -25 * np.abs(v).max() / total[..., None]
    return 2.0 ** -11 * np.abs(ref) + (2.0 ** -11 + 2 * score + n * 2.0 ** -23) * spread + tiny + 2.0 ** -24


def _check_attention(env, case, seed=0, layers=1, layer=0, rows_extra=0, peak=1.0):
    exq, torch = env
    bits, D, page, KH, H, lens, news, causal, window = case
    c = Case(exq, torch, bits, D, page, KH, lens, news, layers=layers, layer=layer, seed=seed + D).fill()
    T = sum(news)
    q = (c.rng.standard_normal((T + rows_extra, H, D)) * peak).astype(np.float16)
    qd = torch.from_numpy(np.concatenate([q, q], 1)).cuda()[:, :H]               # strided rows
    out = torch.full((H, T + rows_extra, D), 7.0, dtype=torch.float16, device="cuda").transpose(0, 1)
    lse = torch.full((T + rows_extra, H), 7.0, device="cuda")
    scale = 0.9 / np.sqrt(D)
    cache, batch = c.cache(), c.batch(rows=T + rows_extra)
    exq.exq_paged_attn(cache, batch, qd, out=out, scale=scale, causal=causal, window=window, lse=lse, layer=layer)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    got, got_lse = _np(out).astype(np.float64), _np(lse).astype(np.float64)
    scale = float(np.float32(scale))
    for b, (n, L) in enumerate(zip(news, lens)):
        r = slice(c.start[b], c.start[b + 1])
        k, v = c.dense[b]
        qb = q[r].astype(np.float64)
        ref, ref_lse, spread, total = O.attention(qb, k, v, np.arange(L - n, L), scale, causal, window)
        empty = np.isneginf(ref_lse)
        assert np.array_equal(np.isneginf(got_lse[r]), empty)
        assert np.all(got[r][empty] == 0)
        if empty.all():
            continue
        assert np.isfinite(got[r]).all()
        tol = _bound(ref, spread, total, qb, k, v, scale, L, D)
        off = np.abs(got[r] - ref)
        assert np.all(off <= tol), (b, off.max(), (off / tol).max())
        big = np.abs(qb).sum(-1).max() * np.abs(k).max() * scale
        lse_tol = (D + 8) * 2.0 ** -24 * big + L * 2.0 ** -23 + 2.0 ** -20 * np.abs(ref_lse[~empty]) + 2.0 ** -20
        assert np.all(np.abs(got_lse[r][~empty] - ref_lse[~empty]) <= lse_tol)
    assert np.all(got[T:] == 7.0) and np.all(got_lse[T:] == 7.0)                # padding rows
    c.same(cache)
    return c, cache, batch, qd


@pytest.mark.parametrize("case", ATTN, ids=["-".join(map(str, (*c[:5], len(c[5]), max(c[5]), max(c[6]), c[8]))) for c in ATTN])
def test_attention(env, case):
    _check_attention(env, case, rows_extra=2)


@pytest.mark.parametrize("bits", [4, 6, 8, 16])
def test_attention_long_and_peaked(env, bits):
    # enough tokens to be split over blocks; scores of large spread, so that the maximum moves along the sequence
    _check_attention(env, (bits, 128, 64, 2, 8, [9000, 3000, 10], [1, 2, 1], True, 0), seed=1, peak=6.0)


@pytest.mark.parametrize("bits", [4, 16])
def test_attention_chunk_split_and_peaked(env, bits):
    _check_attention(env, (bits, 128, 64, 1, 4, [2500], [70], True, 0), seed=2, layers=3, layer=2, peak=5.0)


@pytest.mark.parametrize("new", [1, 40])
def test_attention_is_deterministic_and_streams(env, new):
    exq, torch = env
    c, cache, batch, q = _check_attention(env, (4, 128, 64, 2, 16, [4000, 900], [new, new], True, 0), seed=4)
    a = exq.exq_paged_attn(cache, batch, q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ws = torch.zeros(exq.exq_paged_attn_workspace_size(cache, batch, 16, q.shape[0]), dtype=torch.uint8, device="cuda")
        for _ in range(3):
            b = exq.exq_paged_attn(cache, batch, q, workspace=ws)
    s.synchronize()
    assert torch.equal(a, b)
    assert int(ws[:65536].sum()) == 0                                              # counters left zero


@pytest.mark.parametrize("new", [1, 48])
def test_attention_in_a_graph_follows_device_lengths(env, new):
    # a captured append + attention replayed with other lengths and pages than it was captured with
    exq, torch = env
    D, KH, H, page = 128, 2, 8, 16
    c = Case(exq, torch, 8, D, page, KH, [300, 200], [new, new], seed=9).fill()
    cache = c.cache()
    T = 2 * new
    q, k, v = (torch.randn(T, h, D, device="cuda").half() for h in (H, KH, KH))
    rope = exq.rope_table(D)
    batch = c.batch(max_kv_len=304)
    out = torch.empty(T, H, D, dtype=torch.float16, device="cuda")
    qo = torch.empty_like(q)
    ws = torch.zeros(exq.exq_paged_attn_workspace_size(cache, batch, H, T), dtype=torch.uint8, device="cuda")

    def step():
        exq.exq_kv_append(cache, batch, k, v, q=q, rope=rope, q_out=qo)
        exq.exq_paged_attn(cache, batch, qo, out=out, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens in ([300, 200], [77, 304], [new, 299]):
        t = np.full_like(c.table, -1)
        ids, at = c.rng.permutation(cache.n_pages), 0
        for b, n in enumerate(lens):
            t[b, :-(-n // page)] = ids[at:at + -(-n // page)]
            at += -(-n // page)
        batch.page_table.copy_(torch.from_numpy(t))
        batch.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        cache.k_scales.nan_to_num_(0.01)
        cache.v_scales.nan_to_num_(0.01)
        g.replay()
        replayed = out.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(replayed, out) and torch.isfinite(out).all()
    assert exq.exq_get_last_device_error() == exq.EXQ_OK


@pytest.mark.parametrize("new", [1, 40])
def test_attention_reports_bad_pages_and_lengths(env, new):
    exq, torch = env
    D, KH, H = 64, 2, 8

    def run(spoil, **bounds):
        c = Case(exq, torch, 4, D, 16, KH, [80, 58], [new, new], seed=3).fill()
        spoil(c)
        q = torch.randn(2 * new, H, D, device="cuda").half()
        exq.exq_paged_attn(c.cache(), c.batch(**bounds), q)
        return exq.exq_get_last_device_error()

    assert run(lambda c: None) == exq.EXQ_OK
    for bad in (-1, -2 ** 31, 2 ** 31 - 1):
        assert run(lambda c: c.table.__setitem__((slice(None), 1), bad)) == exq.EXQ_ERR_INVALID_ARG
    assert run(lambda c: None, max_kv_len=79) == exq.EXQ_ERR_INVALID_ARG
    assert run(lambda c: setattr(c, "lens", [-5, 58]), max_kv_len=80) == exq.EXQ_ERR_INVALID_ARG
    if new > 1:
        assert run(lambda c: None, max_q_len=new - 1) == exq.EXQ_ERR_INVALID_ARG
    assert run(lambda c: c.start.__setitem__(slice(None), [0, 2 * new, new])) == exq.EXQ_ERR_INVALID_ARG
    assert exq.exq_get_last_device_error() == exq.EXQ_OK


def test_attention_refusals(env):
    exq, torch = env
    c = Case(exq, torch, 4, 64, 16, 2, [20], [1], seed=3).fill()
    cache, batch = c.cache(), c.batch()
    q = torch.randn(1, 8, 64, device="cuda").half()
    need = exq.exq_paged_attn_workspace_size(cache, batch, 8, 1)
    assert need >= 65536 and exq.exq_paged_attn_workspace_size(cache, batch, 7, 1) == 0
    for kw in (dict(q=q.float()), dict(q=q[:, :7]), dict(q=q[..., :32]), dict(out=q), dict(window=-1), dict(layer=1),
               dict(scale=float("nan")), dict(lse=torch.zeros(1, 8, device="cuda").half()),
               dict(workspace=torch.zeros(need - 1, dtype=torch.uint8, device="cuda")),
               dict(workspace=torch.zeros(need + 16, dtype=torch.uint8, device="cuda")[16:])):
        with pytest.raises(exq.ExqError):
            exq.exq_paged_attn(**{**dict(cache=cache, batch=batch, q=q), **kw})
    assert exq.exq_get_last_device_error() == exq.EXQ_OK


# ---------------------------------------------------------------- page copies

@pytest.mark.parametrize("bits,D,page,KH,layers,moves", [(4, 64, 16, 1, 3, 2), (6, 128, 256, 2, 2, 4), (8, 256, 32, 3, 1, 5),
                                                         (16, 128, 64, 8, 2, 3), (16, 64, 16, 1, 5, 1)])
def test_copy_pages(env, bits, D, page, KH, layers, moves):
    exq, torch = env
    c = Case(exq, torch, bits, D, page, KH, [page * 2 * moves], [1], layers=layers, seed=bits)
    for i in range(2):
        c.words[i][:] = c.rng.integers(0, 1 << 32, c.words[i].shape, dtype=np.uint32)
        if bits != 16:
            c.scales[i][:] = c.rng.integers(0, 1 << 16, c.scales[i].shape)
    cache = c.cache()
    ids = c.rng.permutation(cache.n_pages)[:2 * moves].astype(np.int32)
    pairs = ids.reshape(moves, 2)
    bad = np.array([[-1, 0], [0, cache.n_pages], [2 ** 31 - 1, 1]], np.int32)
    exq.exq_kv_copy_pages(cache, torch.from_numpy(pairs).cuda())
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    exq.exq_kv_copy_pages(cache, torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    exq.exq_kv_copy_pages(cache, torch.from_numpy(bad).cuda())                     # skipped and reported
    assert exq.exq_get_last_device_error() == exq.EXQ_ERR_INVALID_ARG
    for a in c.words + [s for s in c.scales if s is not None]:
        a[:, pairs[:, 1]] = a[:, pairs[:, 0]]
    c.same(cache)


# ---------------------------------------------------------------- failure detection, types

@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_wait_runs_out_then_recovers(env, bits, new):
    # the producer issues no copies: every wait runs out, the call ends in a timeout, the next one is right again
    exq, torch = env
    c = Case(exq, torch, bits, 128, 64, 2, [700, 90], [new, new], seed=6).fill()
    cache, batch = c.cache(), c.batch()
    q = torch.randn(2 * new, 8, 128, device="cuda").half()
    ws = torch.zeros(exq.exq_paged_attn_workspace_size(cache, batch, 8, 2 * new), dtype=torch.uint8, device="cuda")
    want = exq.exq_paged_attn(cache, batch, q, workspace=ws)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    exq.exq_testing_starve(64)
    try:
        exq.exq_paged_attn(cache, batch, q, workspace=ws)
        assert exq.exq_get_last_device_error() == exq.EXQ_ERR_TIMEOUT
    finally:
        exq.exq_testing_starve(0)
    ws.zero_()
    got = exq.exq_paged_attn(cache, batch, q, workspace=ws)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    assert torch.equal(got, want)


def test_binding_refuses_other_types(env):
    exq, torch = env
    c = Case(exq, torch, 4, 64, 16, 2, [20], [1], seed=3).fill()
    cache, batch = c.cache(), c.batch()
    q = torch.randn(1, 8, 64, device="cuda").bfloat16()
    for call in (lambda: exq.exq_paged_attn(cache, batch, q), lambda: exq.exq_kv_append(cache, batch, q[:, :2], q[:, :2]),
                 lambda: exq.KVCache(cache.k_codes, cache.v_codes, None, cache.v_scales, 4),
                 lambda: exq.KVCache(cache.k_codes, cache.v_codes.float(), cache.k_scales, cache.v_scales, 4),
                 lambda: exq.KVCache(cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales, 16),
                 lambda: exq.KVBatch(batch.q_start, batch.kv_len.float(), batch.page_table, 1, 20),
                 lambda: exq.KVBatch(batch.q_start, batch.kv_len.long(), batch.page_table, 1, 20),
                 lambda: exq.exq_kv_copy_pages(cache, torch.zeros(1, 2, device="cuda"))):
        with pytest.raises(exq.ExqError):
            call()
    assert exq.exq_get_last_device_error() == exq.EXQ_OK


@pytest.mark.parametrize("bits,D", [(4, 128), (8, 64), (16, 128)])
@pytest.mark.parametrize("scale", [-0.05, 0.0])
def test_attention_scales_of_any_sign(env, bits, D, scale):
    exq, torch = env
    for new in (1, 50):
        c = Case(exq, torch, bits, D, 16, 1, [150], [new], seed=D).fill()
        q = c.rng.standard_normal((new, 4, D)).astype(np.float16)
        out = exq.exq_paged_attn(c.cache(), c.batch(), torch.from_numpy(q).cuda(), scale=scale)
        k, v = c.dense[0]
        qd = q.astype(np.float64)
        ref, _, spread, total = O.attention(qd, k, v, np.arange(150 - new, 150), float(np.float32(scale)))
        assert np.all(np.abs(_np(out).astype(np.float64) - ref) <= _bound(ref, spread, total, qd, k, v, scale, 150, D))


def test_attention_of_many_short_and_empty_sequences(env):
    # more sequences than lanes, most of them empty or one tile long: shares that begin and end inside many units
    exq, torch = env
    rng = np.random.default_rng(11)
    lens = [int(n) for n in rng.choice([0, 0, 1, 5, 64, 65, 200], 150)]
    for new in (1, 3):
        _check_attention(env, (4, 64, 16, 1, 6, lens, [min(new, n) for n in lens], True, 0), seed=3)
    _check_attention(env, (16, 64, 16, 1, 6, [n for n in lens[:60]], [min(9, n) for n in lens[:60]], True, 0), seed=3)


@pytest.mark.parametrize("bits,D", [(4, 128), (8, 64), (16, 64)])
def test_attention_of_a_prompt_chunk_among_single_tokens(env, bits, D):
    # every sequence is given as many blocks of rows as the longest one needs, and has one or none
    lens, new = [1, 40, 0, 700, 5, 0, 90, 33], [1, 1, 0, 650, 2, 0, 1, 33]
    for causal in (True, False):
        _check_attention(env, (bits, D, 32, 1, 4, lens, new, causal, 0), seed=D)


@pytest.mark.parametrize("new", [5, 60])
def test_attention_in_the_longest_window(env, new):
    # a window no position reaches, beside more new tokens than cached ones: positions below zero
    _check_attention(env, (4, 64, 16, 1, 2, [2, new, 45], [5, new, 1], True, 2**31 - 1), seed=4)


@pytest.mark.parametrize("bits,D,kvh,heads", [(4, 128, 2, 16), (6, 64, 1, 6), (8, 256, 1, 2), (16, 128, 2, 2)])
def test_attention_of_both_kinds_in_a_graph(env, bits, D, kvh, heads):
    # bounds of a prompt chunk, contents of single tokens and chunks: two launches and one workspace, replayed
    exq, torch = env
    c = Case(exq, torch, bits, D, 16, kvh, [300, 129, 64, 0, 20], [270, 1, 1, 0, 20], seed=8).fill()
    cache, batch = c.cache(), c.batch()
    q = torch.from_numpy(c.rng.standard_normal((292, heads, D)).astype(np.float16)).cuda()
    want = exq.exq_paged_attn(cache, batch, q)
    ws = torch.zeros(exq.exq_paged_attn_workspace_size(cache, batch, heads, 292), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with pytest.raises(exq.ExqError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            exq.exq_paged_attn(cache, batch, q, out=out)                        # captured: a workspace of its own
    with torch.cuda.graph(g):
        exq.exq_paged_attn(cache, batch, q, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
    assert int(ws[:65536].count_nonzero()) == 0 and exq.exq_get_last_device_error() == exq.EXQ_OK
    at = 0
    for b, n in enumerate([270, 1, 1, 0, 20]):
        if n:
            k, v = c.dense[b]
            L = len(k)
            qb = q[at:at + n].double().cpu().numpy()
            scale = float(np.float32(D ** -0.5))
            ref, _, spread, total = O.attention(qb, k, v, np.arange(L - n, L), scale)
            assert np.all(np.abs(_np(want[at:at + n]).astype(np.float64) - ref) <= _bound(ref, spread, total, qb, k, v, scale, L, D))
        at += n


@pytest.mark.parametrize("bits,D", [(4, 128), (16, 128), (8, 64)])
def test_attention_of_units_with_and_without_a_second_tile_of_rows(env, bits, D):
    # 200 and 90 rows a KV head in turn, several units a CTA: the second M tile has rows, has none, has some again
    lens = [int(n) for n in np.random.default_rng(5).integers(100, 700, 24)]
    _check_attention(env, (bits, D, 64, 8, 16, lens, [100 if b % 2 == 0 else 45 for b in range(24)], True, 0), seed=12)


# ---------------------------------------------------------------- values that are not finite

def _check_not_finite(env, case, spoil_cache=None, spoil_q=None, seed=0, values=False):
    """A result that the definition leaves not finite is the same one here, and every other is as near as ever. spoil_cache(c)
    may change words and scales of a filled case; spoil_q(q) some queries. values: of V, where infinity may become NaN,
    and codes make the log-sum-exp NaN too."""
    exq, torch = env
    bits, D, page, KH, H, lens, news, causal, window = case
    c = Case(exq, torch, bits, D, page, KH, lens, news, seed=seed + D).fill()
    q = c.rng.standard_normal((sum(news), H, D)).astype(np.float16)
    if spoil_cache:
        spoil_cache(c)
    if spoil_q:
        spoil_q(q)
    lse = torch.full((sum(news), H), 7.0, device="cuda")
    out = exq.exq_paged_attn(c.cache(), c.batch(), torch.from_numpy(q).cuda(), causal=causal, window=window, lse=lse)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    got, got_lse = _np(out).astype(np.float64), _np(lse).astype(np.float64)
    scale, bad = float(np.float32(D ** -0.5)), 0
    for b, (n, L) in enumerate(zip(news, lens)):
        r = slice(c.start[b], c.start[b + 1])
        k, v = (c.read(b, i) for i in range(2))
        qb = q[r].astype(np.float64)
        with np.errstate(all="ignore"):
            ref, ref_lse, spread, total = O.attention(qb, k, v, np.arange(L - n, L), scale, causal, window)
        finite = lambda a: np.where(np.isfinite(a), a, 0.0)  # noqa: E731
        tol = _bound(finite(ref), finite(spread), np.maximum(finite(total), 1.0), finite(qb), finite(k), finite(v), scale, L, D)
        ok = np.isfinite(ref)
        if values and bits != 16:
            ref_lse = np.where(ok.all(-1), ref_lse, np.nan)                      # such a token's scores are NaN
        if values:
            assert np.array_equal(np.isfinite(got[r]), ok), (b, np.argwhere(np.isfinite(got[r]) != ok)[:8])
        else:
            assert np.array_equal(np.isnan(got[r]), np.isnan(ref)), b
            assert np.array_equal(got[r][np.isinf(ref)], ref[np.isinf(ref)]), b
        off = np.abs(got[r][ok] - ref[ok])
        assert np.all(off <= tol[ok]), (b, off.max())
        assert np.array_equal(np.isnan(got_lse[r]), np.isnan(ref_lse))
        assert np.array_equal(np.isneginf(got_lse[r]), np.isneginf(ref_lse))
        there = np.isfinite(ref_lse)
        big = np.abs(finite(qb)).sum(-1).max() * np.abs(finite(k)).max() * scale   # as in _check_attention
        lse_tol = (D + 8) * 2.0 ** -24 * big + L * 2.0 ** -23 + 2.0 ** -20 * np.abs(ref_lse[there]) + 2.0 ** -20
        assert np.all(np.abs(got_lse[r][there] - ref_lse[there]) <= lse_tol)
        bad += (~ok).sum()
    return bad


def _set_key(c, i, b, pos, head, value):
    """K's (i = 0) or V's (1) group of a cached token: its scale (codes), or one fp16 value."""
    page, slot = c.table[b, pos // c.page], pos % c.page
    if c.bits == 16:
        c.words[i].view(np.float16)[c.layer, page, head, slot, 3] = value
    else:
        c.scales[i].view(np.float16)[c.layer, page, head, slot] = value


# one token and chunks of new ones; sequences of one CTA and of many
NOT_FINITE = [(4, 128, 64, 2, 16, [300, 9000, 40], [1, 1, 1], True, 0), (16, 128, 16, 1, 4, [200, 9000], [2, 2], True, 0),
              (8, 64, 32, 2, 8, [90, 6000], [1, 1], True, 0), (6, 256, 16, 1, 4, [70, 5000], [1, 1], True, 0),
              (4, 128, 64, 1, 8, [150, 2500], [45, 45], True, 0), (16, 64, 16, 2, 8, [140, 2500], [60, 33], True, 0),
              (8, 256, 64, 1, 8, [100, 1500], [20, 40], True, 0), (6, 128, 32, 1, 8, [150, 1200], [50, 45], True, 0)]
NOT_FINITE_IDS = ["-".join(map(str, (*c[:5], max(c[6])))) for c in NOT_FINITE]


@pytest.mark.parametrize("case", NOT_FINITE, ids=NOT_FINITE_IDS)
def test_attention_of_queries_that_are_not_finite(env, case):
    def spoil(q):
        q[0, 1, 5] = np.nan
        q[-1, 2, 7] = np.inf
        q[-1, 0, :] = 60000.0            # finite queries beside them
    assert _check_not_finite(env, case, spoil_q=spoil) > 0


@pytest.mark.parametrize("value", [np.inf, np.nan])
@pytest.mark.parametrize("case", NOT_FINITE, ids=NOT_FINITE_IDS)
def test_attention_of_seen_keys_that_are_not_finite(env, case, value):
    # an infinite score among finite ones: its weight is NaN, or 0 where it is negative; whichever piece of a unit holds it
    def spoil(c):
        for b, L in enumerate(c.lens):
            _set_key(c, 0, b, min(37, L - 1), 0, value)
            _set_key(c, 0, b, L - 1, c.KH - 1, value)
    assert _check_not_finite(env, case, spoil_cache=spoil) > 0


# ---------------------------------------------------------------- V of very different sizes

def _bound_by_row(ref, spread, w, vs, bits, q, k, scale, D):
    """_bound for one row, from what the row sees alone: w its weights (the largest is 1) and vs V's scales. Products below
    fp16's normal range lose 2^-25 of the row's largest product each, times a code."""
    n = w.size
    score = (D + 8) * 2.0 ** -24 * np.abs(q).sum() * np.abs(k).max() * scale
    tiny = n * 2.0 ** -25 * (w * vs).max() * 2.0 ** (bits - 1) / w.sum()
    return 2.0 ** -11 * np.abs(ref) + (2.0 ** -11 + 2 * score + n * 2.0 ** -23) * spread + tiny + 2.0 ** -24


@pytest.mark.parametrize("place", ["later", "before the window", "of no weight"])
@pytest.mark.parametrize("bits,D,new", [(4, 128, 4), (8, 64, 8), (6, 256, 4), (4, 128, 60), (8, 64, 70), (6, 256, 40)])
def test_attention_beside_values_of_another_size(env, bits, D, new, place):
    # V of the tokens is about 2^-8, of one token 2^10: rows that do not see it, or whose weight of it is 2^-50 or less, are as
    # near to their result as if it were not there
    exq, torch = env
    L, window = 210, 100 if place == "before the window" else 0
    c = Case(exq, torch, bits, D, 16, 1, [L], [new], seed=bits + new).fill()
    c.put(0, 1, (c.rng.standard_normal((L, 1, D)) * 2.0 ** -8).astype(np.float16), np.arange(L))
    q = c.rng.standard_normal((new, 1, D)).astype(np.float16)
    q[:] = q[:1] + np.float16(0.125) * q           # queries alike: one key far from all of them
    at = np.array([{"later": L - 2, "before the window": L - new // 2 - window, "of no weight": 130}[place]])
    c.put(0, 1, (c.rng.standard_normal((1, 1, D)) * 2.0 ** 10).astype(np.float16), at)
    if place == "of no weight":
        c.put(0, 0, (q[:1] * np.float16(-60 / (D ** -0.5 * (q[0].astype(np.float64) ** 2).sum()))).astype(np.float16), at)
    out = _np(exq.exq_paged_attn(c.cache(), c.batch(), torch.from_numpy(q).cuda(), window=window)).astype(np.float64)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    k, v = c.read(0, 0)[:, 0], c.read(0, 1)[:, 0]
    vs = c.scales[1].view(np.float16)[0, c.table[0, np.arange(L) // 16], 0, np.arange(L) % 16].astype(np.float64)
    scale, clear = float(np.float32(D ** -0.5)), 0
    for i in range(new):
        pos = L - new + i
        seen = np.arange(max(0, pos - window + 1) if window else 0, pos + 1)
        qi = q[i, 0].astype(np.float64)
        x = k[seen] @ qi * scale
        w = np.exp(x - x.max())
        if at[0] in seen:
            if place != "of no weight":
                continue                            # its own rows are its size
            assert w[seen == at[0]] < 2.0 ** -50
        ref, spread = w @ v[seen] / w.sum(), w @ np.abs(v[seen]) / w.sum()
        tol = _bound_by_row(ref, spread, w, vs[seen], bits, qi, k[seen], scale, D)
        assert np.all(np.abs(out[i, 0] - ref) <= tol), (i, np.abs(out[i, 0] - ref).max(), tol.max())
        clear += 1
    assert clear >= new // 2 - 2 and clear > 0


# beside NOT_FINITE: windows, of one token and of many, and rows that see everything
NOT_FINITE_V = NOT_FINITE + [(4, 128, 16, 2, 16, [300, 9000, 40], [1, 1, 1], True, 70), (16, 128, 16, 1, 4, [200, 900], [3, 2], True, 65),
                             (16, 64, 16, 2, 2, [500, 300], [300, 70], True, 90), (8, 128, 32, 1, 4, [500, 700], [90, 200], True, 33),
                             (16, 256, 16, 1, 4, [130, 700], [5, 3], True, 50), (16, 256, 16, 1, 4, [330, 700], [60, 30], True, 50),
                             (16, 128, 64, 1, 4, [200, 90], [40, 3], False, 0), (6, 64, 64, 1, 4, [200, 90], [40, 3], False, 20)]


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("case", NOT_FINITE_V, ids=["-".join(map(str, (*c[:5], max(c[6]), c[7], c[8]))) for c in NOT_FINITE_V])
def test_attention_of_values_that_are_not_finite(env, case, value):
    # the newest token (seen by the last rows alone), one in the middle of the new ones, one that the window leaves on the
    # way; in the last head one that no row sees, or that all see: rows that do not see one are untouched
    bits, D, page, KH, H, lens, news, causal, window = case

    def spoil(c):
        for b, (L, n) in enumerate(zip(lens, news)):
            for at in {L - 1, L - n // 2 - 1} | ({max(L - n // 2 - window, 0)} if window else set()):
                _set_key(c, 1, b, at, 0, value)
            if window and L - n - window >= 0:
                _set_key(c, 1, b, L - n - window, KH - 1, value)             # just before every row's window
            elif KH > 1:
                _set_key(c, 1, b, 0, KH - 1, value)
    assert _check_not_finite(env, case, spoil_cache=spoil, values=True) > 0


@pytest.mark.parametrize("bits,D,new", [(4, 128, 1), (8, 64, 3), (16, 128, 2), (6, 128, 50), (16, 64, 80), (4, 256, 40)])
def test_attention_beside_slots_that_hold_nan(env, bits, D, new):
    # every token before the window and after the row is NaN, K and V: row by row the same as a sequence without them
    exq, torch = env
    L, window, page = 400, 90, 16
    case = (bits, D, page, 1, 2, [L], [new], True, window)
    c = Case(exq, torch, *case[:4], [L], [new], seed=5).fill()
    q = torch.from_numpy(c.rng.standard_normal((new, 2, D)).astype(np.float16)).cuda()
    want = exq.exq_paged_attn(c.cache(), c.batch(), q, window=window)
    for i in range(2):
        for at in range(0, L - new - window + 1):
            _set_key(c, i, 0, at, 0, np.nan)
    assert torch.equal(exq.exq_paged_attn(c.cache(), c.batch(), q, window=window), want)
    for i in range(2):
        for at in range(L - new + 1, L):
            _set_key(c, i, 0, at, 0, np.nan)
    got = exq.exq_paged_attn(c.cache(), c.batch(), q, window=window)
    assert torch.equal(got[:1], want[:1]) and exq.exq_get_last_device_error() == exq.EXQ_OK


@pytest.mark.parametrize("bits,D,page,new,window", [(4, 128, 16, 1, 100), (8, 64, 32, 3, 70), (16, 128, 16, 2, 130), (6, 256, 16, 1, 33),
                                                    (4, 128, 16, 50, 100), (16, 64, 32, 80, 100), (16, 256, 16, 40, 50), (8, 128, 64, 1, 64),
                                                    (6, 128, 32, 45, 20)])
def test_attention_after_the_pages_before_the_window_are_gone(env, bits, D, page, new, window):
    # pages that lie before every new token's window are not read: their entries name no page
    exq, torch = env
    lens = [400, 333, 77]
    c = Case(exq, torch, bits, D, page, 2, lens, [new] * 3, seed=window).fill()
    q = torch.from_numpy(c.rng.standard_normal((3 * new, 4, D)).astype(np.float16)).cuda()
    want = exq.exq_paged_attn(c.cache(), c.batch(), q, window=window)
    gone = 0
    for b, L in enumerate(lens):
        n = max(0, L - new - window + 1) // page
        for i in range(2):                                       # whoever has the pages now
            c.words[i][:, c.table[b, :n]] = 0x7E007E00
            if bits != 16:
                c.scales[i][:, c.table[b, :n]] = 0x7E00
        c.table[b, :n] = -1
        gone += n
    got = exq.exq_paged_attn(c.cache(), c.batch(), q, window=window)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK and gone > 0
    assert torch.equal(got, want)


def test_append_reports_a_q_start_that_falls(env):
    # every token finds a sequence with room for it, but not its own: nothing is written
    exq, torch = env
    k = torch.randn(20, 2, 64, device="cuda").half()
    for start in ([1, 9, 9, 0, 20], [0, 20, 20, 20, 3], [0, 9, 8, 8, 20]):
        c = Case(exq, torch, 8, 64, 16, 2, [40, 40, 40, 40], [5, 5, 5, 5], seed=3)
        c.start[:] = start
        cache = c.cache()
        exq.exq_kv_append(cache, c.batch(max_q_len=20), k, k)
        assert exq.exq_get_last_device_error() == exq.EXQ_ERR_INVALID_ARG, start
        c.same(cache)


MANY_HEADS = [(4, 128, 64, 1, 64, [500, 77], [1, 1], True, 0), (16, 128, 16, 1, 64, [300], [1], True, 100),
              (8, 64, 32, 2, 142, [90, 200], [1, 3], True, 0), (6, 256, 16, 1, 33, [200], [1], True, 0),
              (4, 64, 16, 1, 40, [3000], [1], True, 0), (16, 256, 64, 1, 24, [150, 70], [1, 1], True, 0),
              (8, 128, 256, 1, 300, [140], [5], True, 70)]


@pytest.mark.parametrize("case", MANY_HEADS, ids=["-".join(map(str, (*c[:5], max(c[6])))) for c in MANY_HEADS])
def test_attention_of_many_query_heads_a_kv_head(env, case):
    # more query heads than a unit of the few-row kernel has rows: several units, or the kernel of many rows for one token
    _check_attention(env, case, seed=21)
