"""Host threads and the default workspace of exq_fp4_gemv and exq_moe, without a GPU: a stand-in for the library looks at what
each call is given. A call is several launches that pass data through the workspace, and the lock of Python is free meanwhile."""
from __future__ import annotations

import threading
import time
import weakref

import pytest
import torch


class OnGpu(torch.Tensor):
    def get_device(self):
        return 0


def on_gpu(*shape, dtype=torch.uint8):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


class Library:
    """Two calls at once with memory of one workspace, or one whose memory is gone before it returns, are faults."""

    def __init__(self, buffers):
        self.buffers, self.inside, self.faults, self.calls, self.lock = buffers, {}, [], 0, threading.Lock()

    def exq_fp4_scale_bytes(self, fmt, rows, K):
        return 512 * -(-rows // 128) * -(-K // (64 if fmt == 1 else 128))

    def exq_fp4_gemv_workspace_size(self, w, M):
        return (6 << 20) * M  # above the least size: more rows let the workspace grow

    exq_moe_workspace_size = exq_fp4_gemv_workspace_size

    def _call(self, ws):
        with self.lock:
            if self.inside.get(ws):
                self.faults.append("two calls at once")
            self.inside[ws] = self.inside.get(ws, 0) + 1
        memory = self.buffers[ws]
        for _ in range(2):
            time.sleep(0.002)
            if memory() is None:
                self.faults.append("the memory is gone")
        with self.lock:
            self.inside[ws] -= 1
            self.calls += 1
        return 0

    def exq_fp4_gemv(self, w, x, M, out, ws, n, stream):
        return self._call(ws)

    def exq_moe(self, layer, x, T, ids, weights, y, ws, n, stream):
        return self._call(ws)

    def exq_get_last_device_error(self, stream):
        return 4  # EXQ_ERR_TIMEOUT


@pytest.fixture
def binding(monkeypatch):
    from quantized_weight_exq_gb300 import exq as mod
    buffers = {}
    empty, streams = torch.empty, threading.local()

    def fake_empty(*a, device=None, **kw):
        t = empty(*a, **kw)
        if str(device).startswith("cuda"):
            buffers[t.data_ptr()] = weakref.ref(t)
        return t

    lib = Library(buffers)
    monkeypatch.setattr(torch, "empty", fake_empty)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(mod, "_lib", lib)
    monkeypatch.setattr(mod, "_stream_ptr", lambda stream, device=None: getattr(streams, "handle", 7))
    monkeypatch.setattr(mod, "_fp4_ws", {})
    assert lib.exq_get_last_device_error(None) == mod.EXQ_ERR_TIMEOUT
    return mod, lib, streams


def _run(workers):
    errors = []

    def guarded(f):
        try:
            f()
        except Exception as e:  # noqa: BLE001  (a thread's is lost otherwise)
            errors.append(e)

    threads = [threading.Thread(target=guarded, args=(w,)) for w in workers]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def _calls(mod):
    w = mod.Fp4Matrix(on_gpu(8, 16), on_gpu(512), 1)
    parts = [mod.Fp4Experts(on_gpu(2, 32, 16), on_gpu(2, 512), 1) for _ in range(3)]
    layer = mod.MoeLayer(*parts, top_k=1)
    half = lambda m: on_gpu(m, 32, dtype=torch.float16)  # noqa: E731
    return (lambda m: mod.exq_fp4_gemv(w, half(m)),
            lambda m: mod.exq_moe(layer, half(m), on_gpu(m, 1, dtype=torch.int32), on_gpu(m, 1, dtype=torch.float32)))


def test_calls_of_threads_on_one_stream(binding):
    mod, lib, _ = binding
    gemv, moe = _calls(mod)
    _run([lambda: [gemv(m) for m in (1, 2, 1, 4, 2)], lambda: [moe(m) for m in (1, 1, 3, 5, 1)], lambda: [gemv(m) for m in (6, 1, 7)]])
    assert lib.calls == 13 and not lib.faults, lib.faults


def test_a_reported_timeout_waits_for_calls(binding):
    mod, lib, _ = binding
    gemv, moe = _calls(mod)

    def ask():
        for _ in range(20):
            assert mod.exq_get_last_device_error() == mod.EXQ_ERR_TIMEOUT
            time.sleep(0.001)

    _run([lambda: [gemv(2) for _ in range(6)], lambda: [moe(1) for _ in range(6)], ask])
    assert lib.calls == 12 and not lib.faults, lib.faults
    mod.exq_get_last_device_error()
    assert not mod._fp4_ws  # what was kept is not used again


def test_calls_on_two_streams_do_not_wait(binding):
    mod, lib, streams = binding
    gemv, _ = _calls(mod)
    met = threading.Barrier(2, timeout=20)
    lib._call = lambda ws: 0 * met.wait()  # both calls are inside at once, or this times out

    def on(handle):
        streams.handle = handle
        gemv(1)

    _run([lambda: on(7), lambda: on(8)])
    assert len(mod._fp4_ws) == 2
