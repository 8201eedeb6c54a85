"""One attention block with quantised weights and a paged, quantised KV cache, from the prompt to the last token:

- the projections are EXL2 layers (exq_quantize_exl2), q, k and v in one grouped call;
- the prompt goes in by chunks: exq_kv_append turns q and k by their positions and writes the pages, exq_paged_attn reads
  them;
- the sequence is forked: the continuations share the prompt's whole pages and copy the page that it ends in;
- the decode steps of all continuations are one CUDA graph, replayed with the lengths it finds on the GPU;
- one continuation ends, its pages are freed and the cache is compacted; the others go on.

    python examples/paged_decode.py [--bits 4] [--prompt 4000] [--forks 8] [--steps 64]

The weights and the inputs are random: the times are those of the path, the values mean nothing.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_weight_exq_gb300 as exq  # noqa: E402


class Attention:
    """The block: its four projections, the cache with the host's page counts, the rotary table."""

    def __init__(self, hidden: int, heads: int, kv_heads: int, D: int, bits: int, pages: int, page_size: int, weight_bits: int,
                 seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def layer(K, N):
            w = torch.randn(K, N, generator=gen, device="cuda").mul_(K ** -0.5).half()
            return exq.exq_quantize_exl2(w, np.full(K // 32, weight_bits, np.uint8))

        self.heads, self.kv_heads, self.D = heads, kv_heads, D
        self.qkv = [layer(hidden, heads * D), layer(hidden, kv_heads * D), layer(hidden, kv_heads * D)]
        self.o = layer(heads * D, hidden)
        self.cache = exq.kv_cache(1, pages, kv_heads, page_size, D, bits)
        self.refs = np.zeros(pages, np.int32)
        self.rope = exq.rope_table(D)

    def forward(self, x, batch, workspace=None, gemv_workspace=None):
        """x fp16 [tokens, hidden], the new tokens of the batch's sequences one after another."""
        T = x.shape[0]
        q, k, v = (torch.empty(T, w.N, dtype=torch.float16, device=x.device) for w in self.qkv)
        if T <= 16:
            exq.exq_gemv_multi(self.qkv, x, [q, k, v], workspace=gemv_workspace)
        else:
            exq.exq_gemm_multi(self.qkv, x, [q, k, v])
        q, k, v = q.view(T, self.heads, self.D), k.view(T, self.kv_heads, self.D), v.view(T, self.kv_heads, self.D)
        exq.exq_kv_append(self.cache, batch, k, v, q=q, rope=self.rope, q_out=q)
        a = exq.exq_paged_attn(self.cache, batch, q, workspace=workspace).view(T, -1)
        y = torch.empty_like(x)
        if T <= 16:
            exq.exq_gemv(self.o, a, y, workspace=gemv_workspace)
        else:
            exq.exq_gemm(self.o, a, y)
        return y


def _dev(a):
    return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32), device="cuda")


def run(hidden=8192, heads=64, kv_heads=8, D=128, bits=4, page_size=256, weight_bits=4, prompt=4000, chunk=2048, forks=8, steps=64,
        seed=0):
    """Returns the block, the inputs and the outputs of the prompt [prompt, hidden] and of the steps [steps, forks, hidden]
    (the first fork's stop at half of them), and the time of a step in ms."""
    if not 2 <= forks <= 16 or steps < 4:
        raise ValueError("two to sixteen continuations (one exq_gemv each step) of four tokens or more")
    own = -(-(prompt + steps) // page_size)  # pages of one whole sequence
    shared = prompt // page_size
    block = Attention(hidden, heads, kv_heads, D, bits, shared + forks * (own - shared) + 1, page_size, weight_bits, seed)
    cache, refs = block.cache, block.refs
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    xp = torch.randn(prompt, hidden, generator=gen, device="cuda").half()
    xs = torch.randn(steps, forks, hidden, generator=gen, device="cuda").half()
    ys = torch.zeros_like(xs)

    # the prompt, chunk by chunk
    ids = exq.exq_pages_alloc(refs, -(-prompt // page_size))
    yp = []
    for t in range(0, prompt, chunk):
        n = min(chunk, prompt - t)
        yp.append(block.forward(xp[t:t + n], exq.KVBatch(_dev([0, n]), _dev([t + n]), _dev(ids[None]), n, t + n)))

    # the continuations: the prompt's pages, shared, and pages of their own for what comes
    table = np.full((forks, own), -1, np.int32)
    for f in range(forks):
        got, pairs = (ids, np.empty((0, 2), np.int32)) if f == 0 else exq.exq_pages_fork(refs, ids, prompt, page_size)
        if len(pairs):
            exq.exq_kv_copy_pages(cache, _dev(pairs))
        table[f] = np.concatenate([got, exq.exq_pages_alloc(refs, own - len(got))])

    def decode(f0, first, last):
        """The steps first .. last - 1 of the continuations from f0 on, whose pages table names: one graph, replayed."""
        rows = forks - f0
        x = torch.empty(rows, hidden, dtype=torch.float16, device="cuda")
        kv_len = torch.full((rows,), prompt + first + 1, dtype=torch.int32, device="cuda")
        batch = exq.KVBatch(_dev(np.arange(rows + 1)), kv_len, _dev(table), 1, prompt + steps)
        # the graph's own workspaces
        zeros = lambda n: torch.zeros(max(n, 1), dtype=torch.uint8, device="cuda")  # noqa: E731
        ws = zeros(exq.exq_paged_attn_workspace_size(cache, batch, heads, rows))
        gws = zeros(max(exq.exq_gemv_multi_workspace_size(block.qkv, rows), exq.exq_gemv_workspace_size(block.o, rows)))
        x.copy_(xs[first, f0:])
        block.forward(x, batch, ws, gws)  # the first step once without the graph: replayed, it writes the same again
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = block.forward(x, batch, ws, gws)
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        for t in range(first, last):
            if t == first + 1:  # the first replay also loads what it launches
                torch.cuda.synchronize()
                begin.record()
            x.copy_(xs[t, f0:])
            graph.replay()
            ys[t, f0:] = y
            kv_len += 1
        end.record()
        torch.cuda.synchronize()
        return begin.elapsed_time(end) / (last - first - 1)

    half = steps // 2
    ms = decode(0, 0, half)
    # the first continuation ends: its pages go, the held ones move to the lowest ids
    exq.exq_pages_free(refs, table[0])
    table = np.ascontiguousarray(table[1:])
    pairs = exq.exq_pages_compact(refs, table)
    if len(pairs):
        exq.exq_kv_copy_pages(cache, _dev(pairs))
    decode(1, half, steps)
    status = exq.exq_get_last_device_error()
    if status != exq.EXQ_OK:
        raise exq.ExqError(status, "paged_decode")
    return block, (xp, xs), (torch.cat(yp), ys), ms, len(pairs)


def main():
    p = argparse.ArgumentParser(description="paged decode of one attention block with quantised weights")
    for name, value in (("hidden", 8192), ("heads", 64), ("kv-heads", 8), ("bits", 4), ("page-size", 256), ("prompt", 4000),
                        ("chunk", 2048), ("forks", 8), ("steps", 64)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    block, _, _, ms, moved = run(**{k: v for k, v in vars(a).items()})
    held = int((block.refs > 0).sum())
    print(f"{a.forks} continuations of {a.prompt} tokens, {a.bits}-bit cache: {ms * 1e3:.0f} us a step in a graph; "
          f"{moved} pages moved, {held} of {block.refs.size} held after the first one ended")


if __name__ == "__main__":
    main()
