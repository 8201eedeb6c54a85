"""Memory that the binding keeps or allocates for a call: workspaces of streams and of captured graphs, results of calls on
another stream than the current one."""
from __future__ import annotations

import numpy as np
import pytest

import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch

    import __graft_entry__
    __graft_entry__.build()
    import quantized_weight_exq_gb300 as exq
    torch.cuda.set_device(0)
    return exq, torch


def _long_sequence(exq, torch, tokens=20000, new=1):
    """A cache of one sequence whose units many CTAs share (a large workspace), its batch and queries."""
    pages = -(-tokens // 64)
    cache = exq.kv_cache(1, pages, 2, 64, 128, 16)
    gen = torch.Generator(device="cuda").manual_seed(3)
    for t in (cache.k_codes, cache.v_codes):
        t.view(torch.float16).copy_(torch.randn(*t.shape[:-1], 128, generator=gen, device="cuda"))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = exq.KVBatch(i32([0, new]), i32([tokens]), i32([list(range(pages))]), new, tokens)
    return cache, batch, torch.randn(new, 16, 128, generator=gen, device="cuda").half()


def _layer(exq, K, N):
    e = synth.exl2_layer(K, N, bits=np.full(K // 32, 4), seed=2)
    qw, off = exq.exq_pack_exl2(e.q, e.bits)
    return exq.exl2_weight(qw, off, e.s, e.perm, K, N)


def test_a_graph_keeps_the_default_workspace_it_was_captured_with(env):
    exq, torch = env
    mod = exq.exq
    w = _layer(exq, 512, 256)
    x = torch.from_numpy(synth.activations(1, 512, seed=1)).cuda()
    y = torch.empty(1, 256, dtype=torch.float16, device="cuda")
    before = mod._gemv_ws.pop(0, None)                   # whatever earlier tests have grown it to
    exq.exq_gemv(w, x, y)
    want = y.clone()
    held = mod._gemv_ws[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        exq.exq_gemv(w, x, y)
    cache, batch, q = _long_sequence(exq, torch)
    assert exq.exq_paged_attn_workspace_size(cache, batch, 16, 1) > held.numel()
    exq.exq_paged_attn(cache, batch, q)
    assert mod._gemv_ws[0] is held                       # attention has its own
    mod._shared_workspace(held.numel() + 1)              # and a larger GEMV leaves the graph's where it is
    assert mod._gemv_ws[0] is not held and any(t is held for t in mod._gemv_ws_outgrown)
    ones = [torch.ones(held.numel(), dtype=torch.uint8, device="cuda") for _ in range(4)]
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    del ones, before


def test_attention_on_several_streams_without_a_workspace(env):
    # each stream has a workspace of its own, zeroed in its order; the streams' calls overlap
    exq, torch = env
    cache, batch, q = _long_sequence(exq, torch)
    want = exq.exq_paged_attn(cache, batch, q)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for rep in range(8):
        for i, s in enumerate(streams):
            if i == 0:
                outs.append(exq.exq_paged_attn(cache, batch, q, stream=s))
            elif i == 1:
                outs.append(exq.exq_paged_attn(cache, batch, q, stream=s.cuda_stream))
            else:
                with torch.cuda.stream(s):
                    outs.append(exq.exq_paged_attn(cache, batch, q))
    outs.append(exq.exq_paged_attn(cache, batch, q, stream=0))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    kept = {k[1]: t for k, t in exq.exq._attn_ws.items()}
    mine = [kept[s.cuda_stream] for s in streams]
    assert len({t.data_ptr() for t in mine}) == 3 and all(int(t[:65536].count_nonzero()) == 0 for t in mine)


def test_attention_refuses_capture_of_the_stream_it_is_given(env):
    exq, torch = env
    cache, batch, q = _long_sequence(exq, torch, tokens=300)
    out = torch.empty_like(q)
    want = exq.exq_paged_attn(cache, batch, q)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    ws = torch.zeros(exq.exq_paged_attn_workspace_size(cache, batch, 16, 1), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        with pytest.raises(exq.ExqError):
            exq.exq_paged_attn(cache, batch, q, out=out)
        with pytest.raises(exq.ExqError):
            exq.exq_paged_attn(cache, batch, q, out=out, stream=s)
        exq.exq_paged_attn(cache, batch, q, out=out, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("what", ["rope", "append", "attention", "dequantize"])
def test_results_on_another_stream_do_not_meet_pending_work_on_this_one(env, what):
    # the current stream still has a write to memory that has been given back: a result that is written on another stream
    # must not be put there
    exq, torch = env
    cache, batch, q = _long_sequence(exq, torch, tokens=256, new=256)
    k, v = (torch.randn(256, 2, 128, device="cuda").half() for _ in range(2))
    rope, pos = exq.rope_table(128), torch.arange(256, dtype=torch.int32, device="cuda")
    codes, scales = exq.exq_kv_quantize(q, 4)
    ws = torch.zeros(exq.exq_paged_attn_workspace_size(cache, batch, 16, 256), dtype=torch.uint8, device="cuda")
    call = {"rope": lambda **kw: exq.exq_rope(q, pos, rope, **kw),
            "append": lambda **kw: exq.exq_kv_append(cache, batch, k, v, q=q, rope=rope, **kw),
            "attention": lambda **kw: exq.exq_paged_attn(cache, batch, q, workspace=ws, **kw),
            "dequantize": lambda **kw: exq.exq_kv_dequantize(codes, scales, 128, 4, **kw)}[what]
    want = call()
    s = torch.cuda.Stream()
    call(stream=s)
    torch.cuda.synchronize()
    for handle in (s, s.cuda_stream):
        gone = torch.empty_like(want)
        torch.cuda._sleep(40_000_000)                    # about 20 ms: the write below is still to come
        gone.fill_(7.0)
        del gone
        got = call(stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(got, want), what


@pytest.mark.parametrize("new", [1, 60])
def test_the_default_workspace_survives_a_timeout(env, new):
    # a call whose waits run out leaves the counters of shared units as it found them: the next one needs no fresh workspace
    exq, torch = env
    cache, batch, q = _long_sequence(exq, torch, tokens=3000, new=new)
    want = exq.exq_paged_attn(cache, batch, q)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    exq.exq_testing_starve(64)
    try:
        exq.exq_paged_attn(cache, batch, q)
        assert exq.exq_get_last_device_error() == exq.EXQ_ERR_TIMEOUT
    finally:
        exq.exq_testing_starve(0)
    kept = exq.exq._attn_ws[0, torch.cuda.current_stream().cuda_stream]
    assert int(kept[:65536].count_nonzero()) == 0
    for _ in range(2):
        assert torch.equal(exq.exq_paged_attn(cache, batch, q), want)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
