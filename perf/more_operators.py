"""Microscaled 4-bit floating point: quantisation, products, and a mixture-of-experts layer for a few tokens.

A matrix [rows, K] holds one e2m1 code (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) for each value, two to
a byte along K, the even one in the low half, and one scale byte for each block along K: "e4m3" = blocks of 16 with an e4m3 scale
and one factor for the whole matrix, "e8m0" = blocks of 32 with a power of two. Scale bytes lie in tiles of 128 rows x 4 blocks:
row r, block j of a tile is byte (r % 32) * 16 + (r / 32) * 4 + j of its 512; the tiles of 128 rows follow one another along K.

Each case is one call, or the two calls, that a program makes. `run` computes it in plain torch operations, or, with `own` set,
through the library's entry points. Sizes are those of the Llama-2-70B and 7B projections (8192 and 28672, 4096 and 11008) and generic ones.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BLOCK = {"e4m3": 16, "e8m0": 32}


# ---------------------------------------------------------------- cases

def _readback(name, rows, K, fmt):
    return {"name": name, "op": "readback", "rows": rows, "K": K, "fmt": fmt}


def _product(name, op, M, N, K, fmt):
    return {"name": name, "op": op, "M": M, "N": N, "K": K, "fmt": fmt}


def _moe(name, T, E, k, K, inner, fmt, renorm):
    return {"name": name, "op": "moe", "T": T, "E": E, "k": k, "K": K, "inner": inner, "fmt": fmt, "renorm": renorm}


def listed():
    return [
        # one token's activations, quantised and read back: latency counts
        _readback("quantise and read, 1 x 8192 e4m3", 1, 8192, "e4m3"),
        # a 70B weight, quantised and read back to see what the format loses of it
        _readback("quantise and read, 28672 x 8192 e8m0", 28672, 8192, "e8m0"),
        # one decoded token through a 7B projection: the smallest product
        _product("few rows, 1 x 4096 x 4096 e4m3", "gemv", 1, 4096, 4096, "e4m3"),
        # one decoded token through the 70B gate projection
        _product("few rows, 1 x 28672 x 8192 e8m0", "gemv", 1, 28672, 8192, "e8m0"),
        # drafted tokens checked together, an odd number of them, through the 7B down projection
        _product("few rows, 13 x 4096 x 11008 e4m3", "gemv", 13, 4096, 11008, "e4m3"),
        # a decode step of 64 sequences: activations quantised, then multiplied; few output tiles
        _product("linear, 64 x 8192 x 8192 e4m3", "linear", 64, 8192, 8192, "e4m3"),
        # a prompt of 1777 tokens through the 7B gate projection, its activations quantised on the way
        _product("linear, 1777 x 11008 x 4096 e8m0", "linear", 1777, 11008, 4096, "e8m0"),
        # a prompt chunk through the 70B gate projection, activations that are quantised already (up shares them): the largest
        _product("product, 2048 x 28672 x 8192 e4m3", "gemm", 2048, 28672, 8192, "e4m3"),
        # ragged in every size: rows, columns and K end inside tiles
        _product("product, 333 x 1000 x 2080 e8m0", "gemm", 333, 1000, 2080, "e8m0"),
        # one decoded token through a few large experts
        _moe("experts, 1 token, 2 of 8 e4m3", 1, 8, 2, 4096, 11008, "e4m3", True),
        # five drafted tokens through many experts
        _moe("experts, 5 tokens, 8 of 128 e4m3", 5, 128, 8, 4096, 1536, "e4m3", True),
        # a decode step of 16 sequences through small experts, weights not normalised over the chosen
        _moe("experts, 16 tokens, 6 of 64 e8m0", 16, 64, 6, 2048, 1408, "e8m0", False),
    ]


def _log(r, lo, hi):
    return int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))


def draw(r):
    op = r.choice(["readback", "gemv", "gemv", "linear", "gemm", "moe", "moe"])
    fmt = r.choice(["e4m3", "e8m0"])
    if op == "readback":
        K = 32 * _log(r, 2, 512)
        return _readback("", _log(r, 1, min(28672, 234000000 // K)), K, fmt)
    if op == "moe":
        E = r.choice([4, 8, 16, 32, 60, 64, 128])
        k, T = r.randrange(1, min(8, E) + 1), r.choice([1, 1, r.randrange(2, 17)])
        K = 32 * _log(r, 8, 128)
        most = min(280000000 // (T * k * K), 800000000 // (E * K), 11008)  # what is chosen, what is held
        return _moe("", T, E, k, K, 32 * _log(r, 2, max(3, most // 32)), fmt, r.random() < 0.5)
    K, N = 32 * _log(r, 2, 512), 8 * _log(r, 8, 3584)
    if op == "gemv":
        return _product("", op, r.choice([1, 1, r.randrange(2, 17)]), N, min(K, 32 * (234000000 // (32 * N))), fmt)
    return _product("", op, _log(r, 1, 2048), N, min(K, 32 * (234000000 // (32 * N))), fmt)


def _held(rows, K, fmt):
    return rows * K // 2 + rows * K // BLOCK[fmt]


def work(case):
    K, fmt = case["K"], case["fmt"]
    if case["op"] == "readback":
        n = case["rows"] * K
        return {"bytes": 4 * n + 2 * _held(case["rows"], K, fmt), "flops": 4 * n}
    if case["op"] == "moe":
        T, E, k, I = case["T"], case["E"], case["k"], case["inner"]
        used = E * (1 - (1 - k / E) ** T)  # experts that some token chooses, of a router without preferences
        return {"bytes": int(used * (2 * _held(I, K, fmt) + _held(K, I, fmt))) + 2 * E * K + 4 * T * K + 8 * T * k,
                "flops": 2 * T * E * K + 6 * T * k * I * K}
    M, N = case["M"], case["N"]
    x = {"gemm": _held(M, K, fmt), "gemv": 2 * M * K, "linear": 2 * M * K + 2 * _held(M, K, fmt)}[case["op"]]
    return {"bytes": x + _held(N, K, fmt) + 2 * M * N, "flops": 2 * M * N * K}


# ---------------------------------------------------------------- inputs

def _tiled(scales):
    """Scale bytes [..., rows, blocks] -> [..., bytes] in tiles, zero where a tile reaches over the matrix."""
    *lead, rows, blocks = scales.shape
    t = torch.zeros(*lead, -(-rows // 128) * 128, -(-blocks // 4) * 4, dtype=torch.uint8, device=DEV)
    t[..., :rows, :blocks] = scales
    t = t.unflatten(-1, (-1, 4)).unflatten(-3, (-1, 4, 32))  # [..., row tile, row / 32, row % 32, column tile, j]
    return t.movedim(-2, -4).transpose(-2, -3).flatten(-5).contiguous()


def _weight(gen, shape, fmt, std):
    """Codes [..., rows, K / 2] and scale tiles of weights as a quantiser leaves them: values of a bell curve, each block's largest near 6."""
    *lead, rows, K = shape
    z = torch.randn(*lead, rows, K, generator=gen, device=DEV, dtype=torch.float16)
    c = torch.bucketize(z.abs() * 2.75, torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV, dtype=torch.float16), out_int32=True)
    c = (c + 8 * (z < 0)).to(torch.uint8)
    codes = c[..., 0::2] | (c[..., 1::2] << 4)
    spread = torch.rand(*lead, rows, K // BLOCK[fmt], generator=gen, device=DEV)
    if fmt == "e4m3":  # of a matrix whose factor puts the largest block at 448
        return codes, _tiled((100 + 348 * spread ** 2).to(torch.float8_e4m3fn).view(torch.uint8))
    return codes, _tiled((127 + math.floor(math.log2(std / 2.75)) + (spread < 0.3)).to(torch.uint8))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    K, fmt = case["K"], case["fmt"]
    s = {"case": case}

    def activations(rows):  # a few channels of a model's activations are much larger than the others
        x = torch.randn(rows, K, generator=gen, device=DEV)
        return (x * (1 + 15 * (torch.rand(K, generator=gen, device=DEV) < 0.01))).half()

    if case["op"] == "moe":
        E, I = case["E"], case["inner"]
        s["x"] = torch.randn(case["T"], K, generator=gen, device=DEV).half()
        s["router"] = (torch.randn(E, K, generator=gen, device=DEV) * 1.5 / math.sqrt(K)).half()
        for part, rows, width in (("gate", I, K), ("up", I, K), ("down", K, I)):
            s[part] = _weight(gen, (E, rows, width), fmt, 1 / math.sqrt(width))
            factor = (0.7 + 0.6 * torch.rand(E, generator=gen, device=DEV)) / (math.sqrt(width) * 2.75 * 200)
            s[part + "_factor"] = factor if fmt == "e4m3" else None
        return s
    # factors are calibrated numbers of no special form; e8m0 has none
    s["x_factor"] = (0.021 + 0.001 * (seed % 7)) if fmt == "e4m3" else 1.0
    if case["op"] == "readback":
        s["x"] = activations(case["rows"])
        return s
    s["w"] = _weight(gen, (case["N"], K), fmt, 1 / math.sqrt(K))
    s["w_factor"] = 1.07 / (math.sqrt(K) * 2.75 * 200) if fmt == "e4m3" else 1.0
    if case["op"] == "gemm":
        s["a"] = _quantise(activations(case["M"]), fmt, s["x_factor"])
    else:
        s["x"] = activations(case["M"])
    return s


# ---------------------------------------------------------------- the plain form

def _quantise(x, fmt, factor):
    """(codes, scale tiles) of fp16 rows. Scales: the largest magnitude of a block over 6 (and the factor), rounded to nearest even,
    at least 2^-9 unless the block is zero; or 2^(floor(log2(largest)) - 2). Codes: value over scale, to nearest even, at most 6."""
    b = x.unflatten(-1, (-1, BLOCK[fmt])).double()  # in 64 bits: quotients next to a border
    most = b.abs().amax(-1, keepdim=True)
    if fmt == "e4m3":
        u = most / (6.0 * factor)
        step = torch.ldexp(torch.ones_like(u), torch.frexp(u)[1].clamp(min=-5) - 4)
        s = (torch.round(u / step) * step).clamp(max=448.0)
        s = torch.where(most > 0, s.clamp(min=2.0 ** -9), 0.0)
        scales = s.float().to(torch.float8_e4m3fn).view(torch.uint8)
        q = b.abs() / torch.where(s > 0, s * factor, 1.0)
    else:
        e = torch.where(most > 0, torch.frexp(most)[1] - 3, -127)
        scales = (e + 127).to(torch.uint8)
        q = torch.ldexp(b.abs(), -e)
    c = ((q > 0.25).byte() + (q >= 0.75) + (q > 1.25) + (q >= 1.75) + (q > 2.5) + (q >= 3.5) + (q > 5)).flatten(-2)
    c = c + 8 * torch.signbit(x).byte()
    return c[..., 0::2] | (c[..., 1::2] << 4), _tiled(scales.squeeze(-1))


def _values(codes, tiles, fmt, rows, K):
    """What codes [..., rows, K / 2] and their scales stand for, apart from the matrix's factor: in 32 bits, exact."""
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    v = torch.stack([e2m1[(codes & 15).int()], e2m1[(codes >> 4).int()]], -1).flatten(-2)
    blocks = K // BLOCK[fmt]
    t = tiles.unflatten(-1, (-(-rows // 128), -(-blocks // 4), 32, 4, 4)).transpose(-3, -4).movedim(-2, -4)
    t = t.flatten(-2).flatten(-4, -2)[..., :rows, :blocks]
    s = t.contiguous().view(torch.float8_e4m3fn).float() if fmt == "e4m3" else torch.exp2(t.float() - 127)
    return (v.unflatten(-1, (blocks, -1)) * s[..., None]).flatten(-2)


def _plain_product(s, a, a_factor):
    case = s["case"]
    w = _values(*s["w"], case["fmt"], case["N"], case["K"])
    return ((a @ w.t()) * (a_factor * s["w_factor"])).half()


def _plain_moe(s):
    """Each token's chosen experts, gathered and multiplied in a batch."""
    case = s["case"]
    T, k, K, I, fmt = case["T"], case["k"], case["K"], case["inner"], case["fmt"]
    x = s["x"].float()
    logits = x @ s["router"].float().t()
    best, ids = torch.sort(logits, dim=-1, descending=True, stable=True)  # ties: the lowest index first
    best, ids = best[:, :k], ids[:, :k]
    top = best[:, :1]
    weights = (best - top).exp()
    weights = weights / (weights.sum(-1, keepdim=True) if case["renorm"] else (logits - top).exp().sum(-1, keepdim=True))

    def chosen(part, rows, width):
        (codes, tiles), factor = s[part], s[part + "_factor"]
        w = _values(codes[ids], tiles[ids], fmt, rows, width)
        return w if factor is None else w.mul_(factor[ids][..., None, None])

    g = (chosen("gate", I, K) @ x[:, None, :, None]).squeeze(-1)
    u = (chosen("up", I, K) @ x[:, None, :, None]).squeeze(-1)
    h = g / (1 + (-g).exp()) * u * weights[..., None]
    y = (chosen("down", K, I) @ h[..., None]).squeeze(-1).sum(1)
    return [y.half(), ids.int(), weights]


def _run_plain(s):
    case = s["case"]
    if case["op"] == "moe":
        return _plain_moe(s)
    if case["op"] == "gemv":
        return _plain_product(s, s["x"].float(), 1.0)
    rows, K, fmt = case.get("rows", case.get("M")), case["K"], case["fmt"]
    a = _values(*(s["a"] if case["op"] == "gemm" else _quantise(s["x"], fmt, s["x_factor"])), fmt, rows, K)
    if case["op"] == "readback":
        return (a * s["x_factor"]).half()
    return _plain_product(s, a, s["x_factor"])


# ---------------------------------------------------------------- the library's operators

def _run_own(s):
    import quantized_weight_exq_gb300 as exq
    case = s["case"]
    fmt = exq.FP4_E4M3 if case["fmt"] == "e4m3" else exq.FP4_E8M0
    if case["op"] == "moe":
        if "layer" not in s:  # the weights' descriptors, which a program keeps beside the weights
            parts = [exq.Fp4Experts(*s[p], fmt, s[p + "_factor"]) for p in ("gate", "up", "down")]
            s["layer"] = exq.MoeLayer(*parts, top_k=case["k"], router=s["router"], renorm=case["renorm"])
        return list(exq.exq_moe(s["layer"], s["x"]))
    if case["op"] == "readback":
        return exq.exq_fp4_dequantize(exq.exq_fp4_quantize(s["x"], fmt, s["x_factor"]))
    if "weight" not in s:
        s["weight"] = exq.Fp4Matrix(*s["w"], fmt, s["w_factor"])
    if case["op"] == "gemv":
        return exq.exq_fp4_gemv(s["weight"], s["x"])
    a = exq.Fp4Matrix(*s["a"], fmt, s["x_factor"]) if case["op"] == "gemm" else exq.exq_fp4_quantize(s["x"], fmt, s["x_factor"])
    return exq.exq_fp4_gemm(a, s["weight"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- from the definition, in 64 bits

def _exact_values(codes, tiles, fmt, rows, K):
    """The matrix in 64 bits, from the bits of each code and the place of each scale byte."""
    c = torch.empty(rows, K, dtype=torch.int32, device=DEV)
    c[:, 0::2], c[:, 1::2] = (codes & 15).int(), (codes >> 4).int()
    e, m = (c >> 1) & 3, c & 1
    v = torch.where(e == 0, 0.5 * m, torch.ldexp(1 + 0.5 * m, e - 1)).double() * (1 - 2 * (c >> 3))
    r, j = torch.arange(rows, device=DEV)[:, None], (torch.arange(K, device=DEV) // BLOCK[fmt])[None]
    across = -(-(K // BLOCK[fmt]) // 4)
    b = tiles[(r // 128 * across + j // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4].int()
    if fmt == "e8m0":
        return torch.ldexp(v, b - 127)
    e, m = b >> 3, b & 7
    return v * torch.where(e == 0, m * 2.0 ** -9, torch.ldexp(1 + m / 8.0, e - 7)).double()


def _exact_rounded(x, fmt, factor):
    """The rows' values after quantisation: the nearest of the format's values, ties to those with an even last bit."""
    def nearest(v, grid):  # grid ascending, its even places the even codes
        grid = torch.tensor(grid, dtype=torch.float64, device=DEV)
        i = torch.searchsorted(grid, v.contiguous()).clamp(1, len(grid) - 1)
        lo, hi = grid[i - 1], grid[i]
        up = (v - lo > hi - v) | ((v - lo == hi - v) & (i % 2 == 0))
        return torch.where(up, hi, lo)

    v = x.double().view(x.shape[0], -1, BLOCK[fmt])
    most = v.abs().amax(-1, keepdim=True)
    if fmt == "e4m3":
        grid = [(m if e == 0 else 8 + m) * 2.0 ** (max(e, 1) - 10) for e in range(16) for m in range(8)][:127]
        s = nearest((most / (6.0 * factor)).clamp(max=448.0), grid)
        s = torch.where(most > 0, s.clamp(min=2.0 ** -9), 0.0) * factor
    else:
        s = torch.exp2(torch.floor(torch.log2(torch.where(most > 0, most, 1.0).float())).double() - 2)
    code = nearest((v.abs() / torch.where(s > 0, s, 1.0)).clamp(max=6.0), [0, 0.5, 1, 1.5, 2, 3, 4, 6])
    return (code * s * torch.where(v < 0, -1.0, 1.0)).view(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    K, fmt = case["K"], case["fmt"]
    if case["op"] == "moe":
        T, k, I = case["T"], case["k"], case["inner"]
        x = s["x"].double()
        logits = torch.einsum("tk,ek->te", x, s["router"].double())
        p = torch.softmax(logits, -1)
        ids = torch.argsort(-logits, dim=-1, stable=True)[:, :k]
        weights = p.gather(1, ids)
        if case["renorm"]:
            weights = weights / weights.sum(-1, keepdim=True)
        y = torch.zeros(T, K, dtype=torch.float64, device=DEV)
        for e in ids.unique().tolist():
            def expert(part, rows, width):
                f = s[part + "_factor"]
                return _exact_values(s[part][0][e], s[part][1][e], fmt, rows, width) * (1.0 if f is None else f[e].double())
            t, slot = (ids == e).nonzero(as_tuple=True)
            h = torch.nn.functional.silu(x[t] @ expert("gate", I, K).T) * (x[t] @ expert("up", I, K).T)
            y.index_add_(0, t, (h @ expert("down", K, I).T) * weights[t, slot][:, None])
        return [y, ids.int(), weights]
    if case["op"] == "readback":
        return _exact_rounded(s["x"], fmt, s["x_factor"])
    w = _exact_values(*s["w"], fmt, case["N"], K) * s["w_factor"]
    if case["op"] == "gemv":
        a = s["x"].double()
    elif case["op"] == "linear":
        a = _exact_rounded(s["x"], fmt, s["x_factor"])
    else:
        a = _exact_values(*s["a"], fmt, case["M"], K) * s["x_factor"]
    return a @ w.T
