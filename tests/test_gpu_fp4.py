"""The microscaled 4-bit format on the GPU against 64-bit references: quantiser and dequantiser bit for bit, products within the
rounding of their sums and results."""
from __future__ import annotations

import numpy as np
import pytest

import oracle as O
from helpers import ulp16

pytestmark = pytest.mark.gpu
FORMATS = [1, 2]


@pytest.fixture(scope="module")
def env():
    import torch

    import __graft_entry__
    __graft_entry__.build()
    import quantized_weight_exq_gb300 as exq
    torch.cuda.set_device(0)
    return exq, torch


def _activations(rng, rows, K, spread=4.0):
    """fp16 rows whose blocks differ in magnitude, some of them zero."""
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-spread, spread + 1, (rows, K // 32))).repeat(32, 1)
    x[rng.random((rows, K // 32)).repeat(32, 1) < 0.03] = 0
    return x.astype(np.float16)


def _quantised(exq, torch, rng, rows, K, fmt, factor=1.0):
    """A matrix of random codes and scales of mixed sizes, and its values."""
    codes = rng.integers(0, 16, (rows, K), dtype=np.uint8)
    if fmt == 1:
        scales = rng.integers(0x20, 0x60, (rows, K // 16), dtype=np.uint8)
    else:
        scales = rng.integers(122, 130, (rows, K // 32), dtype=np.uint8)
    return exq.fp4_matrix(codes, scales, fmt, factor), O.fp4_values(codes, scales, fmt, factor)


def _check_quantised(m, x, fmt, factor):
    codes, scales = O.fp4_quantize(x, fmt, factor)
    rows, K = x.shape
    got = O.fp4_unpack(m.codes.cpu().numpy())
    np.testing.assert_array_equal(m.scales.cpu().numpy(), O.fp4_tile(scales))  # the padding's zeros among them
    np.testing.assert_array_equal(got, codes)
    return codes, scales


def _f32_product(values, factor):
    # code times scale has 6 bits: exact in 32 bits, as in 64; the factor rounds once
    return (values.astype(np.float32) * np.float32(factor)).astype(np.float16)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,K", [(1, 32), (1, 8192), (3, 64), (127, 96), (128, 128), (131, 160), (260, 1056), (700, 2080)])
def test_quantize(env, fmt, rows, K):
    exq, torch = env
    rng = np.random.default_rng(rows + K + fmt)
    x = _activations(rng, rows, K)
    for factor in [1.0, 0.0213, 2.0 ** -7, 3.1e5] if fmt == 1 else [1.0]:
        m = exq.exq_fp4_quantize(torch.from_numpy(x).cuda(), fmt, factor)
        codes, scales = _check_quantised(m, x, fmt, factor)
        back = exq.exq_fp4_dequantize(m).cpu().numpy()
        np.testing.assert_array_equal(back, _f32_product(O.fp4_values(codes, scales, fmt), factor))


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_every_magnitude(env, fmt):
    # every finite fp16 number as a block's largest, the others at and next to its ties
    exq, torch = env
    block = O.FP4_BLOCK[fmt]
    top = np.arange(0x7C00, dtype=np.uint16).view(np.float16)
    x = np.zeros((top.size, block), np.float16)
    x[:, 0] = top
    s = O.fp4_scale_values(O.fp4_quantize(np.repeat(x, 32 // block, 1), fmt)[1], fmt)[:, :1]
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    with np.errstate(over="ignore"):
        near = np.clip(s * ties, 0, 65504).astype(np.float16)
    near = np.minimum(near, top[:, None])
    x[:, 1:8] = near
    x[:, 8:15] = -np.minimum(np.nextafter(near, np.float16(65504)), top[:, None])
    if fmt == 1:
        x = np.concatenate([x, -x], 1)
    factors = [1.0, 0.7, 2.0 ** -3, 2.0 ** -60, 2.0 ** 60] if fmt == 1 else [1.0]
    for factor in factors:
        _check_quantised(exq.exq_fp4_quantize(torch.from_numpy(x).cuda(), fmt, factor), x, fmt, factor)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_what_is_not_finite(env, fmt):
    exq, torch = env
    rng = np.random.default_rng(4)
    x = _activations(rng, 40, 160)
    x[3, 17], x[5, 0], x[9, 159], x[9, 40] = np.inf, -np.inf, np.nan, np.float16(-0.0)
    m = exq.exq_fp4_quantize(torch.from_numpy(x).cuda(), fmt)
    codes, scales = _check_quantised(m, x, fmt, 1.0)
    back = exq.exq_fp4_dequantize(m).cpu().numpy()
    want = _f32_product(O.fp4_values(codes, scales, fmt), 1.0)
    assert np.isnan(want).sum() == 3 * O.FP4_BLOCK[fmt]
    np.testing.assert_array_equal(back, want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_dequantize_every_scale(env, fmt):
    exq, torch = env
    n = 128 if fmt == 1 else 256
    codes = np.tile(np.arange(16, dtype=np.uint8), (n, 4 if fmt == 1 else 2))
    scales = np.repeat(np.arange(n, dtype=np.uint8)[:, None], codes.shape[1] // O.FP4_BLOCK[fmt], 1)
    for factor in [1.0, 0.3, 40000.0] if fmt == 1 else [1.0]:
        back = exq.exq_fp4_dequantize(exq.fp4_matrix(codes, scales, fmt, factor)).cpu().numpy()
        with np.errstate(over="ignore"):
            np.testing.assert_array_equal(back, _f32_product(O.fp4_values(codes, scales, fmt), factor))


def _check_product(y, a, w, extra_roundings):
    """|y - ref| within half a step of fp16 and the sum's roundings: each of about K / 16 + extra additions of partial sums is off by
    at most 2^-23 of the sum of magnitudes (the tensor core may cut instead of rounding)."""
    ref = a @ w.T
    size = np.abs(a) @ np.abs(w).T
    tol = 0.5 * ulp16(ref) * (1 + 2.0 ** -8) + (a.shape[1] / 16 + extra_roundings) * 2.0 ** -23 * size + 2.0 ** -25
    y = y.cpu().numpy().astype(np.float64)
    with np.errstate(over="ignore"):
        big = np.abs(ref) >= 65504
    err = np.where(big, 0, np.abs(y - ref))
    assert np.isfinite(y[~big]).all()
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size} off, by {np.max(err / tol):.3g} times what is allowed"


GEMM_SHAPES = [(1, 8, 32), (1, 128, 64), (5, 8, 96), (128, 256, 256), (129, 264, 288), (300, 1000, 2080), (64, 512, 4096), (17, 1032, 160),
               (513, 136, 1056), (256, 384, 64), (2, 2048, 5152), (390, 520, 512), (128, 8, 8224), (1000, 24, 288),
               # tiles of 256 x 256: fewer than the SM pairs and more, the last ones ragged
               (2000, 2056, 96), (1030, 4104, 544), (300, 9000, 64), (2300, 2312, 352), (257, 20000, 32), (6000, 1288, 1312),
               # up to 128 rows: more tiles of 128 columns than SMs, odd counts of stages
               (128, 40008, 1312), (7, 20488, 2336), (100, 30000, 800), (33, 19464, 256),
               # up to 128 rows, few tiles: shares of k in clusters of two, four and eight
               (64, 8192, 1056), (128, 9600, 2080), (17, 4096, 4128), (50, 4104, 8224), (1, 520, 8192), (112, 1536, 8480), (16, 136, 2048)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
def test_gemm(env, fmt, M, N, K):
    exq, torch = env
    rng = np.random.default_rng(M + N + K + fmt)
    fa, fw = (0.013, 0.37) if fmt == 1 else (1.0, 1.0)
    a, av = _quantised(exq, torch, rng, M, K, fmt, fa)
    w, wv = _quantised(exq, torch, rng, N, K, fmt, fw)
    y = torch.full((M, N), float("nan"), dtype=torch.float16, device="cuda")
    exq.exq_fp4_gemm(a, w, out=y)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    _check_product(y, av, wv, 16)
    assert torch.equal(y, exq.exq_fp4_gemm(a, w))  # the same bits again


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("N,K", [(8, 32), (128, 256), (136, 288), (1000, 2080), (4096, 512), (264, 8224), (40, 64), (2048, 4096)])
@pytest.mark.parametrize("M", [1, 2, 8, 9, 16])
def test_gemv(env, fmt, M, N, K):
    exq, torch = env
    rng = np.random.default_rng(M + N + K + fmt)
    w, wv = _quantised(exq, torch, rng, N, K, fmt, 0.37 if fmt == 1 else 1.0)
    x = _activations(rng, M, K, 2)
    y = torch.full((M, N), float("nan"), dtype=torch.float16, device="cuda")
    xd = torch.from_numpy(x).cuda()
    ws = torch.zeros(exq.exq_fp4_gemv_workspace_size(w, M), dtype=torch.uint8, device="cuda")
    exq.exq_fp4_gemv(w, xd, out=y, workspace=ws)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    _check_product(y, x.astype(np.float64), wv, 160)
    assert not ws[:exq.FP4_COUNTER_BYTES].any()
    assert torch.equal(y, exq.exq_fp4_gemv(w, xd))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(8, 4104, 4384), (6, 4744, 4896), (1, 4744, 9760)])
def test_gemv_of_many_units(env, fmt, M, N, K):
    # CTAs with several units, of two rows of tiles
    exq, torch = env
    rng = np.random.default_rng(M + N + K + fmt)
    w, wv = _quantised(exq, torch, rng, N, K, fmt, 0.37 if fmt == 1 else 1.0)
    x = _activations(rng, M, K, 2)
    y = exq.exq_fp4_gemv(w, torch.from_numpy(x).cuda())
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    _check_product(y, x.astype(np.float64), wv, 160)


@pytest.mark.parametrize("fmt", FORMATS)
def test_small_numbers_in_gemv(env, fmt):
    # fp16 subnormals times the smallest scales: nothing is flushed
    exq, torch = env
    rng = np.random.default_rng(8)
    codes = rng.integers(0, 16, (64, 256), dtype=np.uint8)
    scales = np.full((64, 256 // O.FP4_BLOCK[fmt]), 1, np.uint8)
    x = (rng.integers(-1023, 1024, (3, 256)) * 2.0 ** -24).astype(np.float16)
    if fmt == 1:
        w, v = exq.fp4_matrix(codes, scales, 1, 2.0 ** 20), O.fp4_values(codes, scales, 1, 2.0 ** 20)
        _check_product(exq.exq_fp4_gemv(w, torch.from_numpy(x).cuda()), x.astype(np.float64), v, 16)
    else:  # 2^-126 times fp16: sums below fp16's range are zeros, and a block of 2^0 beside them keeps its own
        scales[:, 3] = 127
        v = O.fp4_values(codes, scales, 2)
        x[:, 96:128] = 1.0
        _check_product(exq.exq_fp4_gemv(exq.fp4_matrix(codes, scales, 2), torch.from_numpy(x).cuda()), x.astype(np.float64), v, 16)


@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_scales_stay_in_their_row(env, fmt):
    exq, torch = env
    rng = np.random.default_rng(5)
    nan = 0x7F if fmt == 1 else 0xFF
    M, N, K = 200, 264, 416
    ca, cw = (rng.integers(0, 16, (n, K), dtype=np.uint8) for n in (M, N))
    sa, sw = (np.full((n, K // O.FP4_BLOCK[fmt]), 0x38 if fmt == 1 else 127, np.uint8) for n in (M, N))
    clean_a, clean_w = exq.fp4_matrix(ca, sa, fmt), exq.fp4_matrix(cw, sw, fmt)
    sa, sw = sa.copy(), sw.copy()
    sa[7, 2], sa[199, -1], sw[100, 0], sw[263, -1] = nan, nan, nan, nan
    a, w = exq.fp4_matrix(ca, sa, fmt), exq.fp4_matrix(cw, sw, fmt)
    want = exq.exq_fp4_gemm(clean_a, clean_w)
    got = exq.exq_fp4_gemm(a, w)
    want[[7, 199]] = float("nan")
    want[:, [100, 263]] = float("nan")
    torch.testing.assert_close(got, want, rtol=0, atol=0, equal_nan=True)
    x = torch.from_numpy(_activations(rng, 9, K, 1)).cuda()
    want = exq.exq_fp4_gemv(clean_w, x)
    want[:, [100, 263]] = float("nan")
    torch.testing.assert_close(exq.exq_fp4_gemv(w, x), want, rtol=0, atol=0, equal_nan=True)
    x[4, 77] = float("nan")                                  # and a row of x keeps its NaN to itself
    want[4] = float("nan")
    torch.testing.assert_close(exq.exq_fp4_gemv(w, x), want, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantise_and_multiply(env, fmt):
    # the calls of a linear layer together; few rows unquantised agree with them within the format's error
    exq, torch = env
    rng = np.random.default_rng(6)
    M, N, K = 16, 512, 1024
    x = _activations(rng, M, K, 1)
    wx = (rng.standard_normal((N, K)) / 32).astype(np.float16)
    factor = float(np.abs(wx).max()) / (6 * 448) if fmt == 1 else 1.0
    w = exq.exq_fp4_quantize(torch.from_numpy(wx).cuda(), fmt, factor)
    fx = 0.01 if fmt == 1 else 1.0
    a = exq.exq_fp4_quantize(torch.from_numpy(x).cuda(), fmt, fx)
    wv = O.fp4_values(*O.fp4_quantize(wx, fmt, factor), fmt, factor)
    av = O.fp4_values(*O.fp4_quantize(x, fmt, fx), fmt, fx)
    _check_product(exq.exq_fp4_gemm(a, w), av, wv, 16)
    _check_product(exq.exq_fp4_gemv(w, torch.from_numpy(x).cuda()), x.astype(np.float64), wv, 16)
    # and through the dequantised weight, rounded once to fp16
    np.testing.assert_array_equal(exq.exq_fp4_dequantize(w).cpu().numpy(), _f32_product(O.fp4_values(*O.fp4_quantize(wx, fmt, factor), fmt), factor))


@pytest.mark.parametrize("fmt", FORMATS)
def test_large_product(env, fmt):
    # more tiles than SMs, K of many stages; the reference in 64 bits on the GPU
    exq, torch = env
    rng = np.random.default_rng(7)
    M, N, K = 1100, 6152, 4128
    a, av = _quantised(exq, torch, rng, M, K, fmt)
    w, wv = _quantised(exq, torch, rng, N, K, fmt)
    y = exq.exq_fp4_gemm(a, w)
    da, dw = torch.from_numpy(av).cuda(), torch.from_numpy(wv).cuda()
    ref, size = (da @ dw.T).cpu().numpy(), (da.abs() @ dw.abs().T).cpu().numpy()
    tol = 0.5 * ulp16(ref) * (1 + 2.0 ** -8) + (K / 16 + 16) * 2.0 ** -23 * size
    err = np.abs(y.cpu().numpy().astype(np.float64) - ref)
    assert (err[np.abs(ref) < 65504] <= tol[np.abs(ref) < 65504]).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_pointer_on_a_16_byte_boundary(env, fmt):
    # contiguous views that begin 16 bytes into their memory
    exq, torch = env
    rng = np.random.default_rng(12)

    def off(t):
        n = 16 // t.element_size()
        buf = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")
        view = buf[n:].view(t.shape)
        view.copy_(t)
        assert view.data_ptr() % 32 == 16
        return view

    for M, N, K in ((5, 40, 96), (300, 264, 416)):
        x = _activations(rng, M, K, 1)
        w, wv = _quantised(exq, torch, rng, N, K, fmt)
        w = exq.Fp4Matrix(off(w.codes), off(w.scales), fmt)
        xd = off(torch.from_numpy(x).cuda())
        q = exq.Fp4Matrix(off(torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda")),
                          off(torch.zeros(exq.exq_fp4_scale_bytes(fmt, M, K), dtype=torch.uint8, device="cuda")), fmt)
        half = lambda *s: off(torch.zeros(s, dtype=torch.float16, device="cuda"))  # noqa: E731
        codes, scales = _check_quantised(exq.exq_fp4_quantize(xd, fmt, out=q), x, fmt, 1.0)
        values = O.fp4_values(codes, scales, fmt)
        np.testing.assert_array_equal(exq.exq_fp4_dequantize(q, out=half(M, K)).cpu().numpy(), _f32_product(values, 1.0))
        _check_product(exq.exq_fp4_gemm(q, w, out=half(M, N)), values, wv, 16)
        rows = min(M, 16)
        _check_product(exq.exq_fp4_gemv(w, off(xd[:rows]), out=half(rows, N)), x[:rows].astype(np.float64), wv, 16)


def test_empty(env):
    exq, torch = env
    x = torch.empty(0, 64, dtype=torch.float16, device="cuda")
    m = exq.exq_fp4_quantize(x, 1)
    assert m.rows == 0 and exq.exq_fp4_dequantize(m).shape == (0, 64)
    w, _ = _quantised(exq, torch, np.random.default_rng(1), 24, 64, 1)
    assert exq.exq_fp4_gemm(m, w).shape == (0, 24)


@pytest.mark.parametrize("fmt", FORMATS)
def test_graph_and_other_stream(env, fmt):
    # the whole chain captured with workspaces of its own, replayed on new inputs; and a call on a stream of its own
    exq, torch = env
    rng = np.random.default_rng(9)
    M, N, K = 11, 264, 1056
    w, wv = _quantised(exq, torch, rng, N, K, fmt)
    x = torch.from_numpy(_activations(rng, M, K, 1)).cuda()
    q = exq.exq_fp4_quantize(x, fmt)
    y1, y2, back = (torch.empty(s, dtype=torch.float16, device="cuda") for s in ((M, N), (M, N), (M, K)))
    ws1 = torch.zeros(exq.exq_fp4_gemv_workspace_size(w, M), dtype=torch.uint8, device="cuda")

    def step():
        exq.exq_fp4_quantize(x, fmt, out=q)
        exq.exq_fp4_dequantize(q, out=back)
        exq.exq_fp4_gemm(q, w, out=y2)
        exq.exq_fp4_gemv(w, x, out=y1, workspace=ws1)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        new = _activations(np.random.default_rng(seed), M, K, 1)
        x.copy_(torch.from_numpy(new))
        y1.fill_(float("nan")), y2.fill_(float("nan"))
        graph.replay()
        _check_product(y1, new.astype(np.float64), wv, 16)
        _check_product(y2, O.fp4_values(*O.fp4_quantize(new, fmt), fmt), wv, 16)
    with pytest.raises(exq.ExqError):  # the default workspace is not a graph's
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            exq.exq_fp4_gemv(w, x, out=y1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = exq.exq_fp4_gemv(w, x, stream=side)
    z2 = exq.exq_fp4_gemm(exq.exq_fp4_quantize(x, fmt, stream=side), w, stream=side)
    side.synchronize()
    assert torch.equal(z, y1) and torch.equal(z2, y2)


def test_refusals(env):
    exq, torch = env
    w, _ = _quantised(exq, torch, np.random.default_rng(1), 24, 64, 1)
    x = torch.zeros(3, 64, dtype=torch.float16, device="cuda")
    h = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")  # noqa: E731
    other, _ = _quantised(exq, torch, np.random.default_rng(1), 24, 64, 2)
    for call in (lambda: exq.exq_fp4_gemv(w, x.float()), lambda: exq.exq_fp4_gemv(w, h(3, 128)[:, ::2]), lambda: exq.exq_fp4_gemv(w, h(3, 96)),
                 lambda: exq.exq_fp4_gemv(w, h(17, 64)), lambda: exq.exq_fp4_gemv(w, h(0, 64)), lambda: exq.exq_fp4_gemv(w, x, out=h(3, 25)),
                 lambda: exq.exq_fp4_gemv(w, x, workspace=torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")),
                 lambda: exq.exq_fp4_gemv(w, x.cpu()), lambda: exq.exq_fp4_quantize(h(3, 48), 1), lambda: exq.exq_fp4_quantize(x, 3),
                 lambda: exq.exq_fp4_quantize(x, 2, 0.5), lambda: exq.exq_fp4_quantize(x, 1, float("nan")), lambda: exq.exq_fp4_quantize(x, 1, out=w),
                 lambda: exq.exq_fp4_dequantize(w, out=h(24, 65)), lambda: exq.exq_fp4_gemm(other, w), lambda: exq.exq_fp4_gemm(w, w, out=h(24, 23)),
                 lambda: exq.Fp4Matrix(w.codes, w.scales[:-512], 1), lambda: exq.Fp4Matrix(w.codes[:, ::2], w.scales, 1),
                 lambda: exq.Fp4Matrix(w.codes.cpu(), w.scales, 1), lambda: exq.Fp4Matrix(w.codes.view(torch.int8), w.scales, 1)):
        with pytest.raises(exq.ExqError):
            call()
    assert exq.exq_get_last_device_error() == exq.EXQ_OK


def test_waits_run_out_then_recover(env):
    exq, torch = env
    rng = np.random.default_rng(2)
    w, wv = _quantised(exq, torch, rng, 512, 2048, 1)
    a, av = _quantised(exq, torch, rng, 100, 2048, 1)
    xv = _activations(rng, 3, 2048, 1)
    x = torch.from_numpy(xv).cuda()
    ws = torch.zeros(exq.exq_fp4_gemv_workspace_size(w, 3), dtype=torch.uint8, device="cuda")
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    for call in (lambda: exq.exq_fp4_gemv(w, x, workspace=ws), lambda: exq.exq_fp4_gemm(a, w)):
        exq.exq_testing_starve(64)
        try:
            call()
            assert exq.exq_get_last_device_error() == exq.EXQ_ERR_TIMEOUT
        finally:
            exq.exq_testing_starve(0)
    ws[:exq.FP4_COUNTER_BYTES].zero_()
    _check_product(exq.exq_fp4_gemv(w, x, workspace=ws), xv.astype(np.float64), wv, 16)
    _check_product(exq.exq_fp4_gemm(a, w), av, wv, 16)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK


def test_default_workspace_after_waits_run_out(env):
    # counters that a call left behind when it gave up are not the next call's
    exq, torch = env
    rng = np.random.default_rng(3)
    w, wv = _quantised(exq, torch, rng, 512, 2048, 1)
    xv = _activations(rng, 3, 2048, 1)
    x = torch.from_numpy(xv).cuda()
    exq.exq_fp4_gemv(w, x)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    exq.exq_testing_starve(64)
    try:
        exq.exq_fp4_gemv(w, x)
        for kept in exq.exq._fp4_ws.values():
            kept[0][:exq.FP4_COUNTER_BYTES].fill_(1)
        assert exq.exq_get_last_device_error() == exq.EXQ_ERR_TIMEOUT
    finally:
        exq.exq_testing_starve(0)
    _check_product(exq.exq_fp4_gemv(w, x), xv.astype(np.float64), wv, 16)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [1, 2, 7, 16])
def test_what_is_not_finite_in_gemv(env, fmt, M):
    # a row of x with an infinity or a NaN has a NaN row of y, at any place of a block and of a unit; no other changes
    exq, torch = env
    rng = np.random.default_rng(M + fmt)
    w, _ = _quantised(exq, torch, rng, 136, 544, fmt)
    x = torch.from_numpy(_activations(rng, M, 544, 1)).cuda()
    clean = exq.exq_fp4_gemv(w, x)
    assert not torch.isnan(clean).any()
    for at, v in ((0, float("inf")), (255, float("nan")), (256, float("-inf")), (543, float("nan"))):
        spoilt, want = x.clone(), clean.clone()
        spoilt[M - 1, at] = v
        want[M - 1] = float("nan")
        torch.testing.assert_close(exq.exq_fp4_gemv(w, spoilt), want, rtol=0, atol=0, equal_nan=True)


def _blocks_at_ties(factor):
    """E4M3 blocks of every fp16 number as the largest, with the numbers at and next to the ties of its scale and factor."""
    top = np.arange(0x7C00, dtype=np.uint16).view(np.float16)
    x = np.zeros((top.size, 16), np.float16)
    x[:, 0] = top
    s = O.fp4_scale_values(O.fp4_quantize(np.repeat(x, 2, 1), 1, factor)[1], 1)[:, :1]
    with np.errstate(over="ignore"):
        near = np.clip(s * factor * [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], 0, 65504).astype(np.float16)
    near = np.minimum(near, top[:, None])
    x[:, 1:8] = near
    x[:, 8:15] = -np.minimum(np.nextafter(near, np.float16(65504)), top[:, None])
    return np.concatenate([x, -x], 1)


@pytest.mark.parametrize("factor", [0.025, 0.0125, 0.05, 0.1, 0.2, 0.3, 1 / 6, 0.7, 1 / 3, 2.5e-5, 1e10, 0.021 + 0.001 * 4])
def test_quantize_with_a_factor_of_64_bits(env, factor):
    # such factors times a scale are, in 64 bits, numbers that fp16 values are ties of: rounded to 32 bits first they are not
    exq, torch = env
    x = _blocks_at_ties(factor)
    m = exq.exq_fp4_quantize(torch.from_numpy(x).cuda(), 1, factor)
    assert m.factor == factor
    codes, scales = _check_quantised(m, x, 1, factor)
    if factor not in (2.5e-5, 1e10):  # (one has no ties, the other 32 bits)
        rounded = O.fp4_quantize(x, 1, float(np.float32(factor)))
        assert (rounded[0] != codes).any() or (rounded[1] != scales).any()  # the test can tell
    np.testing.assert_array_equal(exq.exq_fp4_dequantize(m).cpu().numpy(), _f32_product(O.fp4_values(codes, scales, 1), factor))
    rng = np.random.default_rng(int(factor * 1e4) % 1000)
    x = _activations(rng, 64, 8192)
    _check_quantised(exq.exq_fp4_quantize(torch.from_numpy(x).cuda(), 1, factor, out=None), x, 1, factor)
    out = exq.Fp4Matrix(torch.zeros(64, 4096, dtype=torch.uint8, device="cuda"),
                        torch.zeros(exq.exq_fp4_scale_bytes(1, 64, 8192), dtype=torch.uint8, device="cuda"), 1, factor)
    _check_quantised(exq.exq_fp4_quantize(torch.from_numpy(x).cuda(), 1, out=out), x, 1, factor)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,units", [(2, 10), (3, 6), (4, 5), (5, 4), (6, 3), (7, 2), (8, 2), (3, 8), (6, 4), (7, 3), (8, 3)])
def test_gemv_splits_rows_of_several_units(env, fmt, M, units):
    # few rows that the product's own warps split (a CTA has at most 10 units and 24 rows of units), with several units a CTA: the rows of a unit
    # go to the four warps in turn from unit to unit, and ten units are more than there are stages
    exq, torch = env
    rng = np.random.default_rng(10 * M + fmt)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    K = 13 * 256 - 224
    N = (units * sms - 5) // 13 * 128 - 120
    count = -(-N // 128) * -(-K // 256)
    assert (units - 1) * sms < count <= units * sms and units <= 10 and M * count <= 24 * sms
    w, wv = _quantised(exq, torch, rng, N, K, fmt, 0.37 if fmt == 1 else 1.0)
    x = _activations(rng, M, K, 2)
    xd = torch.from_numpy(x).cuda()
    y = torch.full((M, N), float("nan"), dtype=torch.float16, device="cuda")
    ws = torch.zeros(exq.exq_fp4_gemv_workspace_size(w, M), dtype=torch.uint8, device="cuda")
    exq.exq_fp4_gemv(w, xd, out=y, workspace=ws)
    assert exq.exq_get_last_device_error() == exq.EXQ_OK
    assert not ws[:exq.FP4_COUNTER_BYTES].any()
    _check_product(y, x.astype(np.float64), wv, 160)
