"""Serving over a paged KV cache: rotary positions, the append to the pages, attention over them, and page copies.

Each case is one call that a serving loop makes. `run` computes it in plain torch operations, or, with `own` set, through
the library's entry points. Head counts are those of Llama-2-70B (64 query heads over 8 KV heads, D = 128) and
Llama-2-7B (32 over 32, D = 128), and a generic 16 over 4 with D = 64 or 256. A cache holds, for every (layer, page,
KV head, slot), one group of D values: 16 = fp16 values, 4 / 6 / 8 = the Q4 / Q6 / Q8 codes of the KV codec and one fp16 scale.
"""
import math
import random

import numpy as np
import torch

own = False

HEADS = {"70b": (64, 8, 128), "7b": (32, 32, 128), "d64": (16, 4, 64), "d256": (16, 4, 256)}
DEV = "cuda"


# ---------------------------------------------------------------- cases

def _rope(name, tokens, heads, D, R, layout, scaling, first, grad):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "D": D, "R": R, "layout": layout, "scaling": scaling,
            "first": first, "grad": grad}


def _append(name, model, bits, page, seqs, new, past, layout):
    return {"name": name, "op": "append", "model": model, "bits": bits, "page": page, "seqs": seqs, "new": new, "past": past,
            "layout": layout}


def _attn(name, model, bits, page, seqs, new, ctx, window):
    return {"name": name, "op": "attn", "model": model, "bits": bits, "page": page, "seqs": seqs, "new": new, "ctx": ctx,
            "window": window}


def _copy(name, model, bits, page, layers, pages, moves):
    return {"name": name, "op": "copy", "model": model, "bits": bits, "page": page, "layers": layers, "pages": pages,
            "moves": moves}


def listed():
    return [
        # one decoded token's 64 query heads, far into a long context: latency counts
        _rope("rope, one token", 1, 64, 128, 128, "half", "yarn", 120001, False),
        # the gradient at a prompt's queries, interleaved pairs on half of each head
        _rope("rope gradient, 8000 tokens", 8000, 64, 128, 64, "interleaved", "bands", 0, True),
        # one decode step of 64 sequences: the new token of each goes into a Q4 cache
        _append("append, decode step Q4", "70b", 4, 256, 64, 1, 255, "half"),
        # the chunks of prompts of 4 sequences, some of them short, into a Q8 cache
        _append("append, prompt chunks Q8", "70b", 8, 256, 4, 2048, 777, "half"),
        # attention of one token over a short context: the smallest call of a chat
        _attn("decode, one sequence, 500 tokens Q4", "70b", 4, 256, 1, 1, 500, 0),
        # a decode step of 32 sequences of mixed lengths
        _attn("decode, 32 sequences, up to 8192 tokens Q4", "70b", 4, 256, 32, 1, 8192, 0),
        # one sequence with a very long context
        _attn("decode, one sequence, 131072 tokens Q8", "70b", 8, 256, 1, 1, 131072, 0),
        # drafted tokens checked together, small pages, one KV head a few query heads
        _attn("check 5 tokens, 16 sequences, up to 5000 tokens Q6", "d64", 6, 16, 16, 5, 5000, 0),
        # a chunk of a long prompt over what the cache has of it
        _attn("prompt chunk 2048 over 16000 tokens Q4", "70b", 4, 256, 1, 2048, 16000, 0),
        # fresh prompts of mixed lengths, one KV head a query head, unquantised cache, sliding window
        _attn("prompts, 4 sequences, up to 3500 tokens fp16, window", "7b", 16, 64, 4, 3500, 3500, 1024),
        # a sequence forked in every layer: its partly filled last page is copied
        _copy("fork, one page in 80 layers Q4", "70b", 4, 256, 80, 8, 1),
        # compaction of a cache of small fp16 pages
        _copy("compact, 1500 pages in 8 layers fp16", "7b", 16, 16, 8, 4096, 1500),
    ]


def _log(r, lo, hi):
    return int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))


def draw(r):
    op = r.choice(["rope", "append", "attn", "attn", "attn", "copy"])
    model = r.choice(["70b", "70b", "7b", "d64", "d256"])
    heads, kv, D = HEADS[model]
    bits, page = r.choice([4, 4, 6, 8, 16]), r.choice([16, 32, 64, 128, 256])
    if op == "rope":
        R = r.choice([D, D, D // 2, D // 4])
        return _rope("", _log(r, 1, 512000 // heads), heads, D, R, r.choice(["half", "interleaved"]),
                     r.choice(["none", "linear", "yarn", "bands"]), _log(r, 1, 1000000) - 1, r.random() < 0.3)
    if op == "append":
        new = r.choice([1, 1, _log(r, 2, 2048)])
        seqs = _log(r, 1, 256) if new == 1 else _log(r, 1, max(1, 8192 // new))
        return _append("", model, bits, page, seqs, new, _log(r, 1, 900) - 1, r.choice(["half", "interleaved"]))
    if op == "copy":
        one = 2 * kv * page * D * bits // 8  # bytes of a page in one layer
        layers = _log(r, 1, 80)
        moves = _log(r, 1, max(1, min(2000, 2800000000 // (one * layers))))
        return _copy("", model, bits, page, layers, 2 * moves + r.randrange(1, 9), moves)
    kind = r.choice(["decode", "decode", "check", "chunk"])
    window = r.choice([0, 0, 0, _log(r, 64, 4096)])
    if kind == "decode":
        seqs = _log(r, 1, 64)
        most = 1000000000 // (kv * D * bits // 4 * seqs)
        return _attn("", model, bits, page, seqs, 1, _log(r, 1, max(2, min(131072, most))), window)
    if kind == "check":
        seqs = _log(r, 1, 32)
        most = 400000000 // (kv * D * bits // 4 * seqs)
        return _attn("", model, bits, page, seqs, r.randrange(2, 17), _log(r, 20, max(21, min(32768, most))), window)
    new = _log(r, 17, 2048)
    most = 1000000000000 // (4 * heads * D * new)  # multiplications of the scores and of the sum over values
    seqs = r.choice([1, 1, 2, 3])
    return _attn("", model, bits, page, seqs, new, new + _log(r, 1, max(2, min(32768, most // seqs))) - 1, window)


def _lengths(case):
    """(new tokens, cached tokens with them) of each sequence: ragged over a batch, from the case alone."""
    B, new = case["seqs"], case["new"]
    r = random.Random("%d %d %d" % (B, new, case.get("ctx", case.get("past", 0))))
    if case["op"] == "append":
        q = [new if i == 0 or new == 1 else r.randint(1, new) for i in range(B)]
        return q, [n + r.randint(0, case["past"]) for n in q]
    kv = [case["ctx"] if i == 0 else r.randint(1, case["ctx"]) for i in range(B)]
    return [min(new, n) for n in kv], kv


def _group_bytes(D, bits):
    return D * 2 if bits == 16 else D * bits // 8 + 2


def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * case["D"]
        return {"bytes": 4 * n + 4 * case["tokens"], "flops": 3 * case["tokens"] * case["heads"] * case["R"]}
    heads, kv, D = HEADS[case["model"]]
    group = _group_bytes(D, case["bits"])
    if case["op"] == "copy":
        return {"bytes": 2 * case["moves"] * case["layers"] * 2 * kv * case["page"] * group, "flops": 0}
    q, length = _lengths(case)
    T = sum(q)
    if case["op"] == "append":  # q, k, v in; q and the groups out
        return {"bytes": T * D * 2 * (2 * heads + 2 * kv) + T * 2 * kv * group, "flops": 3 * T * (heads + kv) * D}
    seen, pairs = 0, 0
    for n, L in zip(q, length):
        w = case["window"] or L + 1
        seen += L - max(0, L - n + 1 - w)  # tokens that some row sees
        first = L - n + 1                  # tokens that row 0 sees without a window; row i sees min(first + i, w)
        full = min(n, max(0, w - first + 1))
        pairs += full * first + full * (full - 1) // 2 + (n - full) * w
    return {"bytes": 2 * seen * kv * group + 4 * T * heads * D, "flops": 4 * pairs * heads * D}


# ---------------------------------------------------------------- inputs

def _inv_freq(R, scaling):
    """Radians a position of each pair and the factor on cos and sin: base 10000, stretched eightfold where scaled."""
    f = 10000.0 ** (-np.arange(0, R, 2, dtype=np.float64) / R)
    if scaling == "linear":
        return f / 8.0, 1.0
    if scaling == "yarn":  # turns over 4096 tokens: 32 and more keep their frequency, 1 and fewer are stretched
        at = lambda turns: R * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), R - 1)
        ramp = np.clip((np.arange(R // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
        return f / 8.0 * ramp + f * (1 - ramp), 0.1 * math.log(8.0) + 1.0
    if scaling == "bands":  # wavelengths under 4096 / 4 keep theirs, those over 4096 are stretched
        turns = 4096 * f / (2 * math.pi)
        mix = np.clip((turns - 1.0) / (4.0 - 1.0), 0, 1)
        return (1 - mix) * f / 8.0 + mix * f, 1.0
    return f, 1.0


def _table(R, scaling):
    f, gain = _inv_freq(R, scaling)
    steps = np.round(f / (2 * math.pi) * 2.0 ** 64).astype(np.uint64)  # turns a position, in units of 2^-64
    return {"freq": torch.from_numpy(f).to(DEV), "steps": torch.from_numpy(steps.view(np.int64)).to(DEV), "R": R, "gain": gain}


def _pack(u, bits):
    """Codes (uint8 [..., D]) as the codec's words, int32 [..., D * bits / 32]: code i at bits [i bits, (i + 1) bits)."""
    if bits == 8:
        b = u
    elif bits == 4:
        b = u[..., 0::2] | (u[..., 1::2] << 4)
    else:
        c = u.unflatten(-1, (-1, 4))
        b = torch.stack([c[..., 0] | (c[..., 1] << 6), (c[..., 1] >> 2) | (c[..., 2] << 4), (c[..., 2] >> 4) | (c[..., 3] << 2)],
                        -1).flatten(-2)
    return b.contiguous().view(torch.int32)


def _codes(words, bits):
    b = words.view(torch.uint8)
    if bits == 8:
        return b
    if bits == 4:
        return torch.stack([b & 15, b >> 4], -1).flatten(-2)
    b = b.unflatten(-1, (-1, 3))
    return torch.stack([b[..., 0] & 63, (b[..., 0] >> 6) | ((b[..., 1] & 15) << 2), (b[..., 1] >> 4) | ((b[..., 2] & 3) << 4),
                        b[..., 2] >> 2], -1).flatten(-2)


def _quantise(x, bits):
    """(codes, scales) of fp16 groups [..., D], as the codec defines them."""
    top = 2 ** (bits - 1) - 1
    f = x.float()
    s = (f.abs().amax(-1) / torch.full((), float(top), device=f.device)).half()  # a true division: by a number torch multiplies
    q = torch.where(s[..., None] > 0, torch.round(f / s.float()[..., None]), 0.0).nan_to_num(0.0).clamp(-top - 1, top)
    return (q + 2 ** (bits - 1)).to(torch.uint8), s


def _values(words, scales, bits):
    """What the groups stand for, in 32 bits (exact: at most 8 + 11 significant bits)."""
    if bits == 16:
        return words.view(torch.float16).float()
    return (_codes(words, bits).float() - 2 ** (bits - 1)) * scales.float()[..., None]


def _pool(gen, shape, D, bits):
    """Cached groups [layers, pages, heads, slots]: keys or values as a model leaves them, some channels larger."""
    x = torch.randn(*shape, D, generator=gen, device=DEV)
    x *= 1 + 3 * (torch.rand(shape[2], 1, D, generator=gen, device=DEV) < 0.05)
    x = x.half()
    if bits == 16:
        return x.view(torch.int32), None
    u, s = _quantise(x, bits)
    return _pack(u, bits), s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=gen, device=DEV).half()  # noqa: E731
    s = {"case": case}
    if case["op"] == "rope":
        s["x"] = randn(case["tokens"], case["heads"], case["D"])
        s["pos"] = torch.arange(case["tokens"], dtype=torch.int32, device=DEV) + (case["first"] + seed % 97)
        s["rope"] = _table(case["R"], case["scaling"])
        return s
    heads, kv, D = HEADS[case["model"]]
    bits, page = case["bits"], case["page"]
    if case["op"] == "copy":
        s["layers"], s["pages"] = case["layers"], case["pages"]
        order = torch.randperm(case["pages"], generator=gen, device=DEV).int()
        s["pairs"] = torch.stack([order[:case["moves"]], order[case["moves"]:2 * case["moves"]]], 1).contiguous()
    else:
        q, length = _lengths(case)
        s["T"], s["max_q"], s["max_kv"] = sum(q), max(q), max(length)
        start = np.concatenate([[0], np.cumsum(q)])
        s["q_start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
        s["kv_len"] = torch.tensor(length, dtype=torch.int32, device=DEV)
        need = [-(-n // page) for n in length]
        s["layers"], s["pages"] = 1, sum(need) + 3
        ids = torch.randperm(s["pages"], generator=gen, device=DEV).int()
        table = torch.full((len(q), max(need)), -1, dtype=torch.int32, device=DEV)  # -1: no page there
        has = torch.arange(max(need), device=DEV)[None] < torch.tensor(need, device=DEV)[:, None]
        table[has] = ids[:sum(need)]
        s["page_table"] = table
        qkv = randn(s["T"], heads + 2 * kv, D)  # one projection's output; its parts are strided views
        s["q"] = qkv[:, :heads]
        if case["op"] == "append":
            s["k"], s["v"] = qkv[:, heads:heads + kv], qkv[:, heads + kv:]
            s["rope"] = _table(D, "none")
    shape = (s["layers"], s["pages"], kv, page)
    (s["k_codes"], s["k_scales"]), (s["v_codes"], s["v_scales"]) = _pool(gen, shape, D, bits), _pool(gen, shape, D, bits)
    return s


# ---------------------------------------------------------------- the plain form

def _cos_sin(pos, rope):
    angle = pos.double()[:, None] * rope["freq"]  # in 64 bits: far positions
    return (angle.cos() * rope["gain"]).float(), (angle.sin() * rope["gain"]).float()


def _rotate(x, pos, rope, layout, grad=False):
    R = rope["R"]
    c, s = (t[:, None] for t in _cos_sin(pos, rope))
    s = -s if grad else s
    f = x[..., :R].float()
    a, b = (f[..., :R // 2], f[..., R // 2:]) if layout == "half" else (f[..., 0::2], f[..., 1::2])
    y = (a * c - b * s, b * c + a * s)
    y = torch.cat(y, -1) if layout == "half" else torch.stack(y, -1).flatten(-2)
    return torch.cat([y.half(), x[..., R:]], -1)


def _token_places(s):
    """(sequence, index in its new tokens, position) of each new token."""
    t = torch.arange(s["T"], dtype=torch.int32, device=DEV)
    seq = torch.searchsorted(s["q_start"], t, right=True) - 1
    i = t - s["q_start"][seq]
    return seq, i, s["kv_len"][seq] - (s["q_start"][seq + 1] - s["q_start"][seq]) + i


def _plain_append(s):
    case = s["case"]
    bits, page = case["bits"], case["page"]
    seq, _, pos = _token_places(s)
    at = s["page_table"][seq, (pos // page).long()].long(), slice(None), (pos % page).long()  # [T, kv, ...] of a layer
    out = [_rotate(s["q"], pos, s["rope"], case["layout"])]
    for new, words, scales in ((_rotate(s["k"], pos, s["rope"], case["layout"]), s["k_codes"], s["k_scales"]),
                               (s["v"], s["v_codes"], s["v_scales"])):
        if bits == 16:
            words.view(torch.float16)[0][at] = new
            out.append(words.view(torch.float16))
        else:
            u, sc = _quantise(new, bits)
            words[0][at], scales[0][at] = _pack(u, bits), sc
            out.append(_values(words, scales, bits).half())
    return out


def _plain_attn(s):
    case = s["case"]
    heads, kv, D = HEADS[case["model"]]
    B, G, mq = case["seqs"], heads // kv, s["max_q"]
    table = s["page_table"].clamp(min=0).long()
    seq, i, pos = _token_places(s)
    q = torch.zeros(B, mq, heads, D, device=DEV)
    q[seq, i.long()] = s["q"].float()
    q = q.view(B, mq, kv, G, D).transpose(1, 2).reshape(B, kv, mq * G, D)

    def dense(words, scales):  # [B, kv, L, D]
        f = _values(words[0][table], None if scales is None else scales[0][table], case["bits"])
        return f.transpose(1, 2).reshape(B, kv, -1, D)

    p = q @ dense(s["k_codes"], s["k_scales"]).transpose(2, 3)
    p *= 1 / math.sqrt(D)
    L = p.shape[-1]
    t = torch.arange(L, device=DEV)
    n = s["q_start"][1:] - s["q_start"][:-1]
    row = (s["kv_len"] - n)[:, None] + torch.arange(mq * G, device=DEV) // G  # position of each row
    hidden = t > torch.minimum(row, s["kv_len"][:, None] - 1)[..., None]
    if case["window"]:
        hidden |= t <= row[..., None] - case["window"]
    p.masked_fill_(hidden[:, None], -math.inf)
    p -= p.amax(-1, keepdim=True).clamp(min=-1e30)
    p.exp_()
    total = p.sum(-1, keepdim=True)
    y = (p @ dense(s["v_codes"], s["v_scales"])) / total.clamp(min=1e-30)
    y = y.view(B, kv, mq, G, D).transpose(1, 2).reshape(B, mq, heads, D)
    return y[seq, i.long()].half()


def _plain_copy(s):
    src, dst = s["pairs"][:, 0].long(), s["pairs"][:, 1].long()
    buffers = [b for b in (s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"]) if b is not None]
    for b in buffers:
        b[:, dst] = b[:, src]
    return _copied(buffers, s["case"]["bits"])


def _copied(buffers, bits):
    return [b.view(torch.float16) if bits == 16 else b for b in buffers]


# ---------------------------------------------------------------- the library's operators

def _run_own(s):
    import quantized_weight_exq_gb300 as exq
    case = s["case"]
    rope = None
    if "rope" in s:
        rope = exq.Rope(s["rope"]["steps"], s["rope"]["R"],
                        exq.ROPE_HALF if case["layout"] == "half" else exq.ROPE_INTERLEAVED, s["rope"]["gain"])
    if case["op"] == "rope":
        return exq.exq_rope(s["x"], s["pos"], rope, grad=case["grad"])
    cache = exq.KVCache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"], case["bits"])
    if case["op"] == "copy":
        exq.exq_kv_copy_pages(cache, s["pairs"])
        return _copied([b for b in (s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"]) if b is not None], case["bits"])
    batch = exq.KVBatch(s["q_start"], s["kv_len"], s["page_table"], s["max_q"], s["max_kv"])
    if case["op"] == "attn":
        return exq.exq_paged_attn(cache, batch, s["q"], window=case["window"])
    q = exq.exq_kv_append(cache, batch, s["k"], s["v"], q=s["q"], rope=rope)
    if case["bits"] == 16:
        return [q, s["k_codes"].view(torch.float16), s["v_codes"].view(torch.float16)]
    D = q.shape[-1]
    shape = (*s["k_scales"].shape, D)
    return [q, exq.exq_kv_dequantize(s["k_codes"], s["k_scales"], D, case["bits"]).view(shape),
            exq.exq_kv_dequantize(s["v_codes"], s["v_scales"], D, case["bits"]).view(shape)]


def run(state):
    if own:
        return _run_own(state)
    return {"rope": lambda s: _rotate(s["x"], s["pos"], s["rope"], s["case"]["layout"], s["case"]["grad"]),
            "append": _plain_append, "attn": _plain_attn, "copy": _plain_copy}[state["case"]["op"]](state)


# ---------------------------------------------------------------- from the definition, in 64 bits

def _exact_rotate(x, pos, rope, layout, grad=False):
    """Each pair as a complex number times gain e^(+-i angle)."""
    R = rope["R"]
    turn = torch.polar(torch.full((), rope["gain"], dtype=torch.float64, device=DEV).expand(pos.numel(), R // 2).contiguous(),
                       (pos.double()[:, None] * rope["freq"]) * (-1 if grad else 1))
    y = x.double().clone()
    first, second = ((slice(0, R // 2), slice(R // 2, R)) if layout == "half" else (slice(0, R, 2), slice(1, R, 2)))
    z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_group(words, scales, bits, D):
    """Cached groups' values, bit by bit."""
    if bits == 16:
        return words.view(torch.float16).double()
    at = torch.arange(D * bits, device=words.device)
    bit = (words.long()[..., at // 32] >> (at % 32)) & 1
    u = (bit.unflatten(-1, (D, bits)) << torch.arange(bits, device=words.device)).sum(-1)
    return (u - 2 ** (bits - 1)).double() * scales.double()[..., None]


def exact(case, seed):
    if case["op"] == "copy":
        return None  # nothing is computed
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rotate(s["x"], s["pos"], s["rope"], case["layout"], case["grad"])
    heads, kv, D = HEADS[case["model"]]
    bits, page = case["bits"], case["page"]
    qs, length = _lengths(case)
    starts = np.concatenate([[0], np.cumsum(qs)]).tolist()
    if case["op"] == "append":
        pools = []
        for words, scales in ((s["k_codes"], s["k_scales"]), (s["v_codes"], s["v_scales"])):
            pools.append(torch.cat([_exact_group(words[:, i:i + 8], None if bits == 16 else scales[:, i:i + 8], bits, D)
                                    for i in range(0, s["pages"], 8)], 1))
        rotated = []
        for b, (n, L) in enumerate(zip(qs, length)):
            a = slice(starts[b], starts[b + 1])
            pos = torch.arange(L - n, L, device=DEV)
            rotated.append(_exact_rotate(s["q"][a], pos, s["rope"], case["layout"]))
            for pool, new in zip(pools, (_exact_rotate(s["k"][a], pos, s["rope"], case["layout"]).half(), s["v"][a])):
                y = new.double()
                if bits != 16:
                    top = 2.0 ** (bits - 1) - 1
                    sc = (y.abs().amax(-1, keepdim=True) / top).half().double()
                    y = torch.clamp(torch.round(y / torch.where(sc > 0, sc, 1.0)), -top - 1, top) * sc
                pages = s["page_table"][b][(pos // page)].long()
                pool[0, pages, :, pos % page] = y
        return [torch.cat(rotated), *pools]
    if work(case)["flops"] > 2e12 or work(case)["bytes"] > 2e9:
        return None
    out = torch.zeros(starts[-1], heads, D, dtype=torch.float64, device=DEV)
    for b, (n, L) in enumerate(zip(qs, length)):
        pages = s["page_table"][b, :-(-L // page)].long()
        t = torch.arange(L, device=DEV)
        for h in range(kv):
            def cached(words, scales):
                got = [_exact_group(words[0, pages[i:i + 64], h], None if bits == 16 else scales[0, pages[i:i + 64], h], bits, D)
                       for i in range(0, len(pages), 64)]
                return torch.cat(got).reshape(-1, D)[:L]
            k, v = cached(s["k_codes"], s["k_scales"]), cached(s["v_codes"], s["v_scales"])
            for i in range(0, n, 256):
                rows = range(i, min(i + 256, n))
                q = s["q"][starts[b] + i:starts[b] + rows[-1] + 1, h * (heads // kv):(h + 1) * (heads // kv)].double()
                x = torch.einsum("igd,td->igt", q, k) / math.sqrt(D)
                at = torch.arange(rows[0], rows[-1] + 1, device=DEV)[:, None] + (L - n)
                seen = (t <= at) & ((t > at - case["window"]) if case["window"] else (t >= 0))
                w = torch.softmax(torch.where(seen[:, None], x, -math.inf), -1)
                out[starts[b] + i:starts[b] + rows[-1] + 1, h * (heads // kv):(h + 1) * (heads // kv)] = torch.einsum("igt,td->igd", w, v)
    return out
