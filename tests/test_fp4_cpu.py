"""The microscaled 4-bit format and the expert layer on the host: packer, sizes, argument checks, and the plan of the even
division of units that the streaming kernel uses."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

import oracle as O


@pytest.fixture(scope="module")
def exq():
    import quantized_weight_exq_gb300 as exq
    return exq


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("rows,K", [(1, 32), (8, 64), (127, 96), (128, 128), (129, 160), (300, 544)])
def test_pack(exq, fmt, rows, K):
    rng = np.random.default_rng(rows * K + fmt)
    codes = rng.integers(0, 16, (rows, K), dtype=np.uint8)
    scales = rng.integers(0, 128 if fmt == 1 else 256, (rows, K // O.FP4_BLOCK[fmt]), dtype=np.uint8)
    packed, tiles = exq.exq_pack_fp4(codes, scales, fmt)
    assert tiles.size == exq.exq_fp4_scale_bytes(fmt, rows, K) == 512 * -(-rows // 128) * -(-K // (4 * O.FP4_BLOCK[fmt]))
    np.testing.assert_array_equal(packed, O.fp4_pack(codes))
    np.testing.assert_array_equal(tiles, O.fp4_tile(scales))
    np.testing.assert_array_equal(O.fp4_unpack(packed), codes)
    np.testing.assert_array_equal(O.fp4_untile(tiles, rows, K // O.FP4_BLOCK[fmt]), scales)


def test_pack_refuses(exq):
    ok = np.zeros((8, 64), np.uint8), np.zeros((8, 4), np.uint8)
    exq.exq_pack_fp4(*ok, 1)
    bad_code, bad_scale = ok[0].copy(), ok[1].copy()
    bad_code[7, 63], bad_scale[7, 3] = 16, 0x80
    for codes, scales, fmt in ((bad_code, ok[1], 1), (ok[0], bad_scale, 1), (*ok, 2), (*ok, 3), (np.zeros((8, 48), np.uint8), np.zeros((8, 3), np.uint8), 1)):
        with pytest.raises(exq.ExqError) as e:
            exq.exq_pack_fp4(codes, scales, fmt)
        assert e.value.status == exq.EXQ_ERR_INVALID_ARG
    exq.exq_pack_fp4(ok[0], np.full((8, 2), 0xFF, np.uint8), 2)  # any e8m0 byte is a scale


@pytest.mark.parametrize("fmt,rows,K", [(0, 8, 64), (3, 8, 64), (1, 0, 64), (1, 8, 0), (1, 8, 48), (2, -1, 64)])
def test_scale_bytes_of_nothing(exq, fmt, rows, K):
    assert exq.exq_fp4_scale_bytes(fmt, rows, K) == 0


def test_oracle_rounding():
    # every tie of the code and what lies next to it, scale 1: a block's 6 fixes it
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    want = [0, 2, 2, 4, 4, 6, 6]
    for fmt, block in O.FP4_BLOCK.items():
        x = np.zeros((3, block), np.float16)
        x[:, 0] = 6 if fmt == 1 else 4
        x[0, 1:8], x[1, 1:8], x[2, 1:8] = ties, np.nextafter(np.float16(ties), np.float16(0)), -np.nextafter(np.float16(ties), np.float16(9))
        codes, scales = O.fp4_quantize(x, fmt)
        assert (O.fp4_scale_values(scales, fmt)[0] == 1).all()
        assert codes[0, 1:8].tolist() == want
        assert codes[1, 1:8].tolist() == [0, 1, 2, 3, 4, 5, 6] and codes[2, 1:8].tolist() == [9, 10, 11, 12, 13, 14, 15]


def _call(name, *args):
    from quantized_weight_exq_gb300 import exq as mod
    return getattr(mod._lib, name)(*[ctypes.byref(a) if isinstance(a, ctypes.Structure) else a for a in args])


def _matrix(exq, **kw):
    base = dict(format=1, rows=64, K=128, factor=0.5, codes=0x10000, scales=0x20000)
    return exq.exq_fp4_matrix(*[{**base, **kw}[f] for f, _ in exq.exq_fp4_matrix._fields_])


MATRIX_BAD = [dict(format=0), dict(format=3), dict(rows=-1), dict(K=0), dict(K=48), dict(K=-32), dict(factor=0.0), dict(factor=-1.0),
              dict(factor=float("nan")), dict(factor=float("inf")), dict(factor=2.0 ** -61), dict(factor=2.0 ** 61),
              dict(format=2, factor=0.5), dict(codes=None), dict(scales=None), dict(codes=0x10008), dict(scales=0x20008)]


def test_quantisers_validate_on_host(exq):
    bad = exq.EXQ_ERR_INVALID_ARG
    for kw in MATRIX_BAD:
        assert _call("exq_fp4_quantize", 0x30000, _matrix(exq, **kw), None) == bad, kw
        assert _call("exq_fp4_dequantize", _matrix(exq, **kw), 0x30000, None) == bad, kw
    for x in (None, 0x30008):
        assert _call("exq_fp4_quantize", x, _matrix(exq), None) == bad
        assert _call("exq_fp4_dequantize", _matrix(exq), x, None) == bad
    assert _call("exq_fp4_quantize", 0x30000, None, None) == bad and _call("exq_fp4_dequantize", None, 0x30000, None) == bad
    for kw in (dict(rows=0x7FFFFF01), dict(rows=0x7FFFFFFF), dict(K=0x7FFFFF20), dict(K=0x7FFFFFE0)):  # past 32 bits, in whole tiles
        assert _call("exq_fp4_quantize", 0x30000, _matrix(exq, **kw), None) == exq.EXQ_ERR_UNSUPPORTED, kw
        assert _call("exq_fp4_dequantize", _matrix(exq, **kw), 0x30000, None) == exq.EXQ_ERR_UNSUPPORTED, kw
        assert _call("exq_fp4_gemm", _matrix(exq, **kw), _matrix(exq), 0x50000, None) == exq.EXQ_ERR_UNSUPPORTED, kw
    empty = _matrix(exq, rows=0, codes=None, scales=None)
    assert _call("exq_fp4_quantize", None, empty, None) == exq.EXQ_OK
    assert _call("exq_fp4_dequantize", empty, None, None) == exq.EXQ_OK


def test_gemm_validates_on_host(exq):
    bad = exq.EXQ_ERR_INVALID_ARG

    def call(a={}, w={}, y=0x50000):
        return _call("exq_fp4_gemm", _matrix(exq, **{"rows": 5, **a}), _matrix(exq, **w), y, None)

    for kw in MATRIX_BAD:
        assert call(a=kw) == bad and call(w=kw) == bad, kw
    assert call(a=dict(format=2, factor=1.0)) == bad and call(a=dict(K=256)) == bad
    assert call(w=dict(rows=0)) == bad and call(w=dict(rows=12)) == bad
    assert call(y=None) == bad and call(y=0x50008) == bad
    assert call(a=dict(rows=0, codes=None, scales=None), y=None) == exq.EXQ_OK


def test_gemv_validates_on_host(exq):
    bad = exq.EXQ_ERR_INVALID_ARG

    def call(w={}, x=0x30000, M=1, y=0x50000):
        return _call("exq_fp4_gemv", _matrix(exq, **w), x, M, y, None, 0, None)

    for kw in MATRIX_BAD:
        assert call(w=kw) == bad, kw
    assert call(w=dict(rows=0)) == bad and call(w=dict(rows=12)) == bad and call(M=0) == bad and call(M=-1) == bad
    assert call(x=None) == bad and call(x=0x30008) == bad and call(y=None) == bad and call(y=0x50002) == bad
    assert call(M=17) == exq.EXQ_ERR_UNSUPPORTED and call(w=dict(rows=4194184)) == exq.EXQ_ERR_UNSUPPORTED
    assert _call("exq_fp4_gemv_workspace_size", _matrix(exq), 17) == 0 and _call("exq_fp4_gemv_workspace_size", _matrix(exq), 0) == 0


def _layer(exq, gate={}, up={}, down={}, **kw):
    part = lambda rows, K, more: exq.exq_fp4_experts(*[{**dict(format=1, n_experts=8, rows=rows, K=K, codes=0x10000, scales=0x20000,  # noqa: E731
                                                               factors=0x30004), **more}[f] for f, _ in exq.exq_fp4_experts._fields_])
    rest = {**dict(router=0x40000, top_k=2, renorm=1, act=0), **kw}
    return exq.exq_moe_layer(part(96, 64, gate), part(96, 64, up), part(64, 96, down), rest["router"], rest["top_k"], rest["renorm"], rest["act"])


def test_moe_validates_on_host(exq):
    bad = exq.EXQ_ERR_INVALID_ARG

    def call(T=1, x=0x50000, ids=0x60004, weights=0x70004, y=0x80000, **kw):
        layer = _layer(exq, **kw)
        assert T <= 16 or _call("exq_moe_workspace_size", layer, T) == 0
        return _call("exq_moe", layer, x, T, ids, weights, y, None, 0, None)

    each = [dict(format=0), dict(format=2), dict(n_experts=7), dict(n_experts=0), dict(rows=95), dict(rows=0), dict(K=80), dict(codes=None),
            dict(scales=None), dict(codes=0x10008), dict(scales=0x20004), dict(factors=0x30002)]
    for kw in each:
        for part in ("gate", "up", "down"):
            assert call(**{part: kw}) == bad, (part, kw)
    all_ = lambda **kw: {p: kw for p in ("gate", "up", "down")}  # noqa: E731
    assert call(**all_(format=2)) == bad                 # factors with e8m0
    assert call(top_k=0) == bad and call(top_k=9) == bad and call(renorm=2) == bad and call(act=2) == bad and call(router=0x40008) == bad
    assert call(T=0) == bad and call(x=None) == bad and call(y=0x80008) == bad and call(ids=None) == bad and call(weights=0x70002) == bad
    assert call(T=17) == exq.EXQ_ERR_UNSUPPORTED and call(**all_(n_experts=513)) == exq.EXQ_ERR_UNSUPPORTED
    assert call(top_k=17, **all_(n_experts=32)) == exq.EXQ_ERR_UNSUPPORTED
    big = 32 * 8191  # 8 tokens of 16 experts: more tiles than counters
    assert call(T=8, top_k=16, gate=dict(n_experts=128, rows=big // 32 * 32), up=dict(n_experts=128, rows=big // 32 * 32),
                down=dict(n_experts=128, K=big // 32 * 32)) == exq.EXQ_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors(exq):
    import torch
    z = lambda *s, dtype=torch.uint8: torch.zeros(*s, dtype=dtype)  # noqa: E731
    for call in (lambda: exq.Fp4Matrix(z(8, 32), z(512), 1), lambda: exq.Fp4Experts(z(2, 8, 32), z(2, 512), 1),
                 lambda: exq.exq_fp4_quantize(z(8, 64, dtype=torch.float16), 1)):
        with pytest.raises(exq.ExqError) as e:
            call()
        assert e.value.status == exq.EXQ_ERR_INVALID_ARG


def test_units_have_one_owner():
    # CTA b of `ctas` has units [b n / ctas, (b + 1) n / ctas); the owner of unit u is ((u + 1) ctas - 1) / n
    rng = np.random.default_rng(1)
    for n in [1, 2, 151, 152, 153, 500, 512, 7168, *rng.integers(1, 100000, 40).tolist()]:
        ctas = min(n, 152)
        start = [b * n // ctas for b in range(ctas + 1)]
        assert start[0] == 0 and start[-1] == n and all(a < b for a, b in zip(start, start[1:]))
        u = np.arange(n, dtype=np.int64)
        owner = ((u + 1) * ctas - 1) // n
        np.testing.assert_array_equal(owner, np.searchsorted(start, u, side="right") - 1)


def test_factor_has_64_bits(exq):
    # the caller's number, not the nearest of 32 bits: 0.025 * 1.25 is 2^-5 in 64 bits only
    assert exq.exq_fp4_matrix(1, 1, 32, 0.025, None, None).factor == 0.025
    x = np.zeros((1, 32), np.float16)
    x[0, :16:2], x[0, 1] = 0.0390625, 0.1875                     # a tie (1.25 * 2^-5) of a block whose scale is 1.25
    codes, scales = O.fp4_quantize(x, 1, 0.025)
    assert O.fp4_scale_values(scales, 1)[0, 0] == 1.25 and codes[0, 0] == 2
    codes, _ = O.fp4_quantize(x, 1, np.nextafter(0.025, 0))      # the next number down: above the tie
    assert codes[0, 0] == 3


@pytest.mark.parametrize("ctas", [1, 2, 148, 152])
def test_units_of_the_kernels_have_one_owner(exq, ctas):
    # the kernels' own arithmetic, on both sides of where it changes to 64 bits (units times CTAs = 2^31)
    lib = exq.exq._lib
    rng = np.random.default_rng(ctas)
    border = 2 ** 31 // ctas
    for n in {ctas, ctas + 1, 3 * ctas - 1, 7168, 8 * 32767, border - 1, border, border + 1, 2 ** 31 - 257, 2 ** 33, *rng.integers(ctas, 10 ** 6, 20).tolist()}:
        start = [lib.exq_testing_first_unit(b, n, ctas) for b in range(ctas + 1)]
        assert start[0] == 0 and start[-1] == n and all(a < b for a, b in zip(start, start[1:]))
        for b in range(ctas):
            for u in {start[b], start[b + 1] - 1, (start[b] + start[b + 1]) // 2}:
                assert lib.exq_testing_unit_owner(u, n, ctas) == b
    assert lib.exq_testing_first_unit(0, ctas - 1, ctas) == -1 and lib.exq_testing_first_unit(ctas + 1, ctas, ctas) == -1
    assert lib.exq_testing_unit_owner(ctas, ctas, ctas) == -1 and lib.exq_testing_unit_owner(0, 0, 0) == -1
