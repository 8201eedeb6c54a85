"""Rotary tables, page bookkeeping and argument checks of the paged KV cache: the host side, without a GPU."""
from __future__ import annotations

import ctypes
from fractions import Fraction

import numpy as np
import pytest

import oracle as O


@pytest.fixture(scope="module")
def exq():
    import __graft_entry__
    __graft_entry__.build()
    import quantized_weight_exq_gb300 as m
    return m


SCALINGS = [dict(), dict(scaling=1, factor=4.0), dict(scaling=2, factor=8.0), dict(base=500000.0),
            dict(scaling=3, factor=8.0, orig_ctx=4096.0, low=1.0, high=32.0),
            dict(scaling=3, factor=1.0, orig_ctx=4096.0), dict(scaling=4, factor=8.0, orig_ctx=8192.0, low=1.0, high=4.0)]


@pytest.mark.parametrize("R", [4, 20, 64, 128])
@pytest.mark.parametrize("kw", SCALINGS)
def test_rope_freqs(exq, R, kw):
    f, gain = exq.exq_rope_freqs(R, **kw)
    rf, rgain = O.rope_freqs(R, **kw)
    np.testing.assert_allclose(f, rf, rtol=1e-13)    # a few fp64 operations and pow
    assert abs(gain - rgain) < 1e-14


def test_rope_freqs_ends(exq):
    # fast pairs keep their frequency, slow ones are stretched by the factor
    plain = 10000.0 ** (-np.arange(64) / 64)
    for kw in SCALINGS[4], SCALINGS[6]:
        f, _ = exq.exq_rope_freqs(128, **kw)
        assert f[0] == plain[0] and f[-1] == pytest.approx(plain[-1] / 8, rel=1e-14)
        assert np.all(f <= plain * (1 + 1e-14)) and np.all(f >= plain / 8 * (1 - 1e-14))


def test_rope_steps_are_turns(exq):
    f, _ = exq.exq_rope_freqs(128)
    f = np.concatenate([f, [0.0, 2 * np.pi, -0.25, 7.5]])
    steps = exq.exq_rope_steps(f)
    assert np.array_equal(steps, O.rope_steps(f))
    for x, s in zip(f, steps):
        t = Fraction(float(x)) / Fraction(2 * np.pi)
        off = abs((t - Fraction(int(s), 1 << 64)) % 1)
        # the fp64 quotient's rounding, and half a unit of the fixed point
        assert min(off, 1 - off) <= Fraction(abs(float(x))) * Fraction(2.0 ** -54) + Fraction(1, 1 << 53)


def test_rope_tables_refuse(exq):
    bad = [dict(R=0), dict(R=7), dict(R=8, base=1.0), dict(R=8, scaling=5), dict(R=8, scaling=1, factor=0.0),
           dict(R=2, scaling=2, factor=2.0), dict(R=8, scaling=3, factor=2.0, orig_ctx=0.0),
           dict(R=8, scaling=4, factor=2.0, orig_ctx=64.0, low=4.0, high=4.0), dict(R=8, base=float("nan"))]
    for kw in bad:
        with pytest.raises(exq.ExqError) as e:
            exq.exq_rope_freqs(**kw)
        assert e.value.status == exq.EXQ_ERR_INVALID_ARG, kw
    with pytest.raises(exq.ExqError):
        exq.exq_rope_steps(np.array([1.0, np.inf]))
    with pytest.raises(exq.ExqError):
        exq.exq_rope_steps(np.array([]))


# ---------------------------------------------------------------- pages

def test_pages_alloc_free(exq):
    refs = np.zeros(6, np.int32)
    assert exq.exq_pages_alloc(refs, 4).tolist() == [0, 1, 2, 3]
    exq.exq_pages_free(refs, [1, 2])
    assert exq.exq_pages_alloc(refs, 3).tolist() == [1, 2, 4]
    before = refs.copy()
    with pytest.raises(exq.ExqError) as e:
        exq.exq_pages_alloc(refs, 2)
    assert e.value.status == exq.EXQ_ERR_FULL and "page" in str(e.value)
    for ids in ([0, 6], [-1], [5], [0, 3, 0]):   # outside, free, named twice but held once
        with pytest.raises(exq.ExqError) as e:
            exq.exq_pages_free(refs, ids)
        assert e.value.status == exq.EXQ_ERR_INVALID_ARG
    assert np.array_equal(refs, before)
    assert exq.exq_pages_alloc(refs, 0).size == 0


@pytest.mark.parametrize("tokens", [0, 1, 15, 16, 17, 32, 40])
def test_pages_fork(exq, tokens):
    refs = np.zeros(8, np.int32)
    ids = exq.exq_pages_alloc(refs, 3)
    child, pairs = exq.exq_pages_fork(refs, ids, tokens, 16)
    whole, part = divmod(tokens, 16)
    assert child[:whole].tolist() == ids[:whole].tolist() and child.size == whole + (part > 0)
    if part:
        assert pairs.tolist() == [[ids[whole], 3]] and child[-1] == 3 and refs[3] == 1
    else:
        assert pairs.size == 0
    assert refs[:3].tolist() == [2 if i < whole else 1 for i in range(3)]
    exq.exq_pages_free(refs, child)
    assert refs.tolist() == [1, 1, 1, 0, 0, 0, 0, 0]


def test_pages_fork_refuses(exq):
    refs = np.array([1, 1], np.int32)
    with pytest.raises(exq.ExqError) as e:
        exq.exq_pages_fork(refs, [0, 1], 20, 16)          # needs a page of its own
    assert e.value.status == exq.EXQ_ERR_FULL and refs.tolist() == [1, 1]
    for ids, n in (([0, 2], 20), ([0], 20), ([0, 1], -1)):
        with pytest.raises(exq.ExqError):
            exq.exq_pages_fork(refs, ids, n, 16)
    refs = np.array([1, 0, 0], np.int32)
    with pytest.raises(exq.ExqError):
        exq.exq_pages_fork(refs, [1], 16, 16)             # a free page cannot be shared
    assert refs.tolist() == [1, 0, 0]


@pytest.mark.parametrize("seed", range(8))
def test_pages_compact(exq, seed):
    rng = np.random.default_rng(seed)
    n = int(rng.integers(1, 60))
    refs = (rng.integers(0, 3, n) * (rng.random(n) < rng.random())).astype(np.int32)
    held = np.flatnonzero(refs)
    tables = rng.choice(np.concatenate([held, [-1]]), (4, 9)).astype(np.int32) if held.size else np.full((4, 9), -1, np.int32)
    pool = rng.integers(0, 1 << 30, n)
    seen, held_by, old_refs = pool[tables], tables >= 0, refs.copy()
    pairs = exq.exq_pages_compact(refs, tables)
    src, dst = pairs[:, 0], pairs[:, 1]
    assert len(set(dst)) == len(dst) and not set(src) & set(dst)
    assert np.all(old_refs[src] > 0) and np.all(old_refs[dst] == 0)
    pool[dst] = pool[src]
    assert np.array_equal(pool[tables][held_by], seen[held_by]) and np.array_equal(tables >= 0, held_by)
    assert np.all(refs[:held.size] > 0) and np.all(refs[held.size:] == 0)
    assert sorted(refs) == sorted(old_refs)


def test_pages_compact_refuses(exq):
    for table in ([3], [1]):   # outside the pool, a free page
        refs, t = np.array([1, 0, 2], np.int32), np.array(table, np.int32)
        with pytest.raises(exq.ExqError):
            exq.exq_pages_compact(refs, t)
        assert refs.tolist() == [1, 0, 2] and t.tolist() == table


# ---------------------------------------------------------------- argument checks of the device calls

def _call(exq, name, *args):
    from quantized_weight_exq_gb300 import exq as mod
    return getattr(mod._lib, name)(*[ctypes.byref(a) if isinstance(a, ctypes.Structure) else a for a in args])


CACHE = dict(bits=4, D=128, n_kv_heads=8, page_size=16, n_pages=10, n_layers=2, k_codes=0x10000, k_scales=0x20000,
             v_codes=0x30000, v_scales=0x40000)
BATCH = dict(n_seqs=2, n_tokens=3, max_q_len=2, max_kv_len=64, max_pages=4, q_start=0x50000, kv_len=0x60000,
             page_table=0x70004)
ROPE = dict(steps=0x80000, R=128, layout=0, gain=1.0)


def _struct(kind, base, kw):
    return kind(*[{**base, **kw}[f] for f, _ in kind._fields_])


def test_rope_validates_on_host(exq):
    rows = exq.exq_rows(0x10000, 1024, 128)

    def call(rope={}, x=rows, n=4, H=8, D=128, pos=0x20004, y=rows, grad=0):
        return _call(exq, "exq_rope", _struct(exq.exq_rope_params, ROPE, rope), x, n, H, D, pos, y, grad, None)

    bad, un = exq.EXQ_ERR_INVALID_ARG, exq.EXQ_ERR_UNSUPPORTED
    assert call(D=132) == un and call(D=520) == un
    for kw in (dict(steps=None), dict(steps=0x80004), dict(R=0), dict(R=130), dict(R=31), dict(layout=2),
               dict(gain=float("nan"))):
        assert call(rope=kw) == bad, kw
    assert call(n=-1) == bad and call(H=-1) == bad and call(grad=2) == bad and call(pos=None) == bad and call(pos=0x20002) == bad
    for r in (exq.exq_rows(None, 1024, 128), exq.exq_rows(0x10008, 1024, 128), exq.exq_rows(0x10000, 1020, 128),
              exq.exq_rows(0x10000, 1024, 132)):
        assert call(x=r) == bad and call(y=r) == bad
    assert call(y=exq.exq_rows(0x10000, 2048, 128)) == bad       # in place with other strides
    assert call(x=None) == bad
    assert call(n=0, x=None, y=None, pos=None) == exq.EXQ_OK and call(H=0) == exq.EXQ_OK


CACHE_BAD = [dict(n_kv_heads=0), dict(n_pages=0), dict(n_layers=0), dict(k_codes=None), dict(v_codes=0x30008),
             dict(k_scales=None), dict(v_scales=0x40002), dict(bits=16)]
CACHE_UNSUPPORTED = [dict(D=96), dict(D=512), dict(bits=5), dict(page_size=8), dict(page_size=48), dict(page_size=512)]
BATCH_BAD = [dict(n_seqs=-1), dict(n_tokens=-1), dict(max_q_len=-1), dict(max_kv_len=65), dict(max_pages=-1),
             dict(q_start=None), dict(kv_len=0x60002), dict(page_table=None)]


def test_append_validates_on_host(exq):
    kv = exq.exq_rows(0x10000, 1024, 128)
    q = exq.exq_rows(0x90000, 8192, 128)

    def call(cache={}, layer=0, batch={}, k=kv, v=kv, rope=_struct(exq.exq_rope_params, ROPE, {}), pos=None, q=q, qo=q, H=64):
        return _call(exq, "exq_kv_append", _struct(exq.exq_kv_cache, CACHE, cache), layer,
                     _struct(exq.exq_kv_batch, BATCH, batch), k, v, rope, pos, q, qo, H, None)

    bad = exq.EXQ_ERR_INVALID_ARG
    for kw in CACHE_BAD:
        assert call(cache=kw) == bad, kw
    for kw in CACHE_UNSUPPORTED:
        assert call(cache=kw) == exq.EXQ_ERR_UNSUPPORTED, kw
    for kw in BATCH_BAD:
        assert call(batch=kw) == bad, kw
    assert call(layer=2) == bad and call(layer=-1) == bad
    assert call(k=None) == bad and call(v=exq.exq_rows(0x10000, 4, 128)) == bad
    assert call(rope=_struct(exq.exq_rope_params, ROPE, dict(R=256))) == bad
    assert call(rope=None) == bad                       # q needs rope
    assert call(rope=None, q=None, qo=None, pos=0x1000) == bad
    assert call(qo=None) == bad and call(H=0) == bad and call(pos=0x1002) == bad
    assert call(qo=exq.exq_rows(0x90000, 8192, 64)) == bad
    assert call(batch=dict(n_tokens=0), k=None, v=None, q=None, qo=None) == exq.EXQ_OK
    assert call(batch=dict(n_seqs=0)) == exq.EXQ_OK


def test_attention_validates_on_host(exq):
    q, out = exq.exq_rows(0x90000, 8192, 128), exq.exq_rows(0xA0000, 8192, 128)

    def call(cache={}, layer=0, batch={}, q=q, H=64, scale=0.1, causal=1, window=0, out=out, lse=None):
        return _call(exq, "exq_paged_attn", _struct(exq.exq_kv_cache, CACHE, cache), layer,
                     _struct(exq.exq_kv_batch, BATCH, batch), q, H, scale, causal, window, out, lse, None, 0, None)

    bad = exq.EXQ_ERR_INVALID_ARG
    for kw in CACHE_BAD:
        assert call(cache=kw) == bad, kw
    for kw in CACHE_UNSUPPORTED:
        assert call(cache=kw) == exq.EXQ_ERR_UNSUPPORTED, kw
    for kw in BATCH_BAD:
        assert call(batch=kw) == bad, kw
    assert call(layer=2) == bad and call(H=0) == bad and call(H=12) == bad and call(causal=2) == bad
    assert call(window=-1) == bad and call(scale=float("inf")) == bad and call(lse=0x1002) == bad
    assert call(q=None) == bad and call(out=q) == bad and call(out=exq.exq_rows(0xA0008, 8192, 128)) == bad
    assert call(batch=dict(n_tokens=0), q=None, out=None) == exq.EXQ_OK


def test_copy_pages_validates_on_host(exq):
    def call(cache={}, pairs=0x1000, n=1):
        return _call(exq, "exq_kv_copy_pages", _struct(exq.exq_kv_cache, CACHE, cache), pairs, n, None)

    for kw in CACHE_BAD:
        assert call(cache=kw) == exq.EXQ_ERR_INVALID_ARG, kw
    assert call(pairs=None) == exq.EXQ_ERR_INVALID_ARG and call(pairs=0x1002) == exq.EXQ_ERR_INVALID_ARG
    assert call(n=-1) == exq.EXQ_ERR_INVALID_ARG and call(n=0, pairs=None) == exq.EXQ_OK


def test_binding_refuses_host_tensors(exq):
    # a tensor that is not on the GPU is an error on the host, before any launch
    import torch
    i32, f16 = torch.int32, torch.float16
    z = lambda *s, dtype=i32: torch.zeros(*s, dtype=dtype)  # noqa: E731
    for call in (lambda: exq.Rope(z(32, dtype=torch.int64), 64), lambda: exq.KVBatch(z(2), z(1), z(1, 4), 1, 64),
                 lambda: exq.KVCache(z(1, 4, 2, 16, 16), z(1, 4, 2, 16, 16), z(1, 4, 2, 16, dtype=f16), z(1, 4, 2, 16, dtype=f16), 4),
                 lambda: exq.exq_rope(z(1, 2, 64, dtype=f16), z(1), None), lambda: exq.exq_kv_copy_pages(None, z(2, 2)),
                 lambda: exq.kv_cache(1, 4, 2, 16, 128, 4, device="cpu")):
        with pytest.raises(exq.ExqError) as e:
            call()
        assert e.value.status == exq.EXQ_ERR_INVALID_ARG


class _Tensor:
    """What the binding asks of a tensor, without a GPU."""

    def __init__(self, shape, dtype, device=0):
        import math
        self.shape, self.dtype, self.device_index, self.is_cuda = tuple(shape), dtype, device, device >= 0
        self._strides = [math.prod(self.shape[i + 1:]) for i in range(len(self.shape))]

    def stride(self):
        return tuple(self._strides)

    def numel(self):
        import math
        return math.prod(self.shape)

    def element_size(self):
        return self.dtype.itemsize

    def is_floating_point(self):
        return self.dtype.is_floating_point

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000

    def get_device(self):
        return self.device_index

    @property
    def device(self):
        import torch
        return torch.device("cuda", self.device_index) if self.is_cuda else torch.device("cpu")


def _batch(exq, device=0, n_tokens=None):
    import torch
    z = lambda *s: _Tensor(s, torch.int32, device)  # noqa: E731
    return exq.KVBatch(z(3), z(2), z(2, 8), 4, 100, n_tokens)


def test_batch_descriptors_of_two_calls_are_their_own(exq):
    # two threads with one batch and other rows: neither passes the other's count
    batch = _batch(exq)
    a = batch.desc(3)
    b = batch.desc(5)
    assert (a.n_tokens, b.n_tokens) == (3, 5) and a.n_seqs == b.n_seqs == 2 and a.max_kv_len == 100
    assert _batch(exq, n_tokens=7).desc(9).n_tokens == 7


def test_binding_refuses_tensors_of_several_devices(exq, monkeypatch):
    # all of a call's tensors are on one device, and it is the current one: anything else is an error before any launch
    import torch
    i32, f16, i64 = torch.int32, torch.float16, torch.int64
    T = _Tensor
    here = [0]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: here[0])

    def cache(d=0, vd=None, sd=None):
        codes = lambda dev: T((1, 8, 2, 16, 8), i32, dev)  # noqa: E731
        scales = lambda dev: T((1, 8, 2, 16), f16, dev)  # noqa: E731
        return exq.KVCache(codes(d), codes(d if vd is None else vd), scales(d), scales(d if sd is None else sd), 4)

    def rope(d=0):
        return exq.Rope(T((32,), i64, d), 64)

    rows = lambda heads, d=0: T((3, heads, 64), f16, d)  # noqa: E731
    pos = lambda d=0: T((3,), i32, d)  # noqa: E731
    bad = [lambda: cache(vd=1), lambda: cache(sd=1),
           lambda: exq.KVBatch(T((3,), i32, 0), T((2,), i32, 1), T((2, 8), i32, 0), 4, 100),
           lambda: exq.KVBatch(T((3,), i32, 0), T((2,), i32, 0), T((2, 8), i32, 1), 4, 100),
           lambda: exq.exq_rope(rows(4, 1), pos(), rope()), lambda: exq.exq_rope(rows(4), pos(1), rope()),
           lambda: exq.exq_rope(rows(4), pos(), rope(1)), lambda: exq.exq_rope(rows(4), pos(), rope(), out=rows(4, 1)),
           lambda: exq.exq_rope(rows(4, -1), pos(), rope()),
           lambda: exq.exq_kv_append(cache(), _batch(exq, 1), rows(2), rows(2)),
           lambda: exq.exq_kv_append(cache(1), _batch(exq), rows(2), rows(2)),
           lambda: exq.exq_kv_append(cache(), _batch(exq), rows(2), rows(2, 1)),
           lambda: exq.exq_kv_append(cache(), _batch(exq), rows(2), rows(2), q=rows(4, 1), rope=rope(), q_out=rows(4)),
           lambda: exq.exq_kv_append(cache(), _batch(exq), rows(2), rows(2), q=rows(4), rope=rope(1), q_out=rows(4)),
           lambda: exq.exq_kv_append(cache(), _batch(exq), rows(2), rows(2), rope=rope(), pos=pos(1)),
           lambda: exq.exq_paged_attn(cache(), _batch(exq), rows(4, 1)),
           lambda: exq.exq_paged_attn(cache(), _batch(exq), rows(4), out=rows(4, 1)),
           lambda: exq.exq_paged_attn(cache(), _batch(exq), rows(4), out=rows(4), lse=T((3, 4), torch.float32, 1)),
           lambda: exq.exq_paged_attn(cache(), _batch(exq), rows(4), out=rows(4), workspace=T((1 << 20,), torch.uint8, -1)),
           lambda: exq.exq_kv_copy_pages(cache(), T((1, 2), i32, 1))]
    for i, call in enumerate(bad):
        with pytest.raises(exq.ExqError) as e:
            call()
        assert e.value.status == exq.EXQ_ERR_INVALID_ARG, i
    here[0] = 1                                          # everything on device 0, the launch would go to 1
    for i, call in enumerate([lambda: exq.exq_rope(rows(4), pos(), rope(), out=rows(4)),
                              lambda: exq.exq_kv_append(cache(), _batch(exq), rows(2), rows(2)),
                              lambda: exq.exq_paged_attn(cache(), _batch(exq), rows(4), out=rows(4)),
                              lambda: exq.exq_kv_copy_pages(cache(), T((1, 2), i32))]):
        with pytest.raises(exq.ExqError) as e:
            call()
        assert e.value.status == exq.EXQ_ERR_INVALID_ARG, i
