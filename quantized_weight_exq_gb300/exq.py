"""Python binding of libexq (ctypes): argument marshalling only.

Every function here forwards to the C ABI in ``include/exq.h`` with the same
name; all arithmetic runs in the library (host packers in C++, device ops in
CUDA kernels). torch is used only to hold device memory and to name the
current CUDA stream. If ``libexq.so`` has not been built, importing this
module raises: there is no fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import threading
from dataclasses import dataclass, field
from pathlib import Path
from typing import Optional

import numpy as np

_LIB_PATH = Path(__file__).resolve().parent / "libexq.so"

EXQ_OK = 0
EXQ_ERR_INVALID_ARG = 1
EXQ_ERR_UNSUPPORTED = 2
EXQ_ERR_CUDA = 3
EXQ_ERR_TIMEOUT = 4
EXQ_ERR_FULL = 5

EXQ_FMT_GPTQ4 = 1
EXQ_FMT_EXL2 = 2
EXQ_FMT_EXL2_QSCALE = 3

FP4_E4M3, FP4_E8M0 = 1, 2
ACT_SILU, ACT_GELU_TANH = 0, 1

ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_SCALE_NONE, ROPE_SCALE_LINEAR, ROPE_SCALE_NTK, ROPE_SCALE_YARN, ROPE_SCALE_BANDS = range(5)

# every symbol include/exq.h declares
EXPORTED = (
    "exq_pack_gptq", "exq_pack_exl2", "exq_pack_exl2_qscale", "exq_exl2_word_rows", "exq_exl2_seg_word_off",
    "exq_dequant", "exq_gemv_workspace_size",
    "exq_gemv", "exq_gemv_multi_workspace_size", "exq_gemv_multi", "exq_gemm_workspace_size", "exq_gemm", "exq_gemm_multi_workspace_size", "exq_gemm_multi", "exq_gemm_noalloc", "exq_status_string",
    "exq_get_last_device_error", "exq_kv_quantize", "exq_kv_dequantize",
    "exq_quantize_exl2", "exq_measure_exl2_workspace_size", "exq_measure_exl2", "exq_solve_exl2_bits",
    "exq_rope_freqs", "exq_rope_steps", "exq_rope", "exq_kv_append", "exq_paged_attn_workspace_size", "exq_paged_attn",
    "exq_kv_copy_pages", "exq_pages_alloc", "exq_pages_free", "exq_pages_fork", "exq_pages_compact",
    "exq_fp4_scale_bytes", "exq_pack_fp4", "exq_fp4_quantize", "exq_fp4_dequantize", "exq_fp4_gemm",
    "exq_fp4_gemv_workspace_size", "exq_fp4_gemv", "exq_moe_workspace_size", "exq_moe",
    "exq_testing_starve", "exq_testing_first_unit", "exq_testing_unit_owner",
)

# most layers one exq_gemv_multi call takes (EXQ_GEMV_MAX_LAYERS)
GEMV_MAX_LAYERS = 4

# size of the static scratch array exq_gemm_noalloc uses (EXQ_NOALLOC_SCRATCH_BYTES)
NOALLOC_SCRATCH_BYTES = 16 << 20


class ExqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class exq_weight(ctypes.Structure):
    _fields_ = [
        ("format", ctypes.c_int32), ("K", ctypes.c_int32), ("N", ctypes.c_int32),
        ("group_size", ctypes.c_int32), ("n_groups", ctypes.c_int32), ("n_word_rows", ctypes.c_int32),
        ("qweight", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("qzeros", ctypes.c_void_p),
        ("perm", ctypes.c_void_p), ("seg_word_off", ctypes.c_void_p),
        ("q_scale", ctypes.c_void_p), ("q_scale_max", ctypes.c_void_p),
    ]


class exq_rope_params(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_void_p), ("R", ctypes.c_int32), ("layout", ctypes.c_int32), ("gain", ctypes.c_double)]


class exq_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class exq_kv_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("bits", "D", "n_kv_heads", "page_size", "n_pages", "n_layers")] + [
        (n, ctypes.c_void_p) for n in ("k_codes", "k_scales", "v_codes", "v_scales")]


class exq_kv_batch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_seqs", "n_tokens", "max_q_len", "max_kv_len", "max_pages")] + [
        (n, ctypes.c_void_p) for n in ("q_start", "kv_len", "page_table")]


class exq_fp4_matrix(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("format", "rows", "K")] + [
        ("factor", ctypes.c_double), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class exq_fp4_experts(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("format", "n_experts", "rows", "K")] + [
        (n, ctypes.c_void_p) for n in ("codes", "scales", "factors")]


class exq_moe_layer(ctypes.Structure):
    _fields_ = [(n, exq_fp4_experts) for n in ("gate", "up", "down")] + [("router", ctypes.c_void_p)] + [
        (n, ctypes.c_int32) for n in ("top_k", "renorm", "act")]


def _load():
    if not _LIB_PATH.exists():
        raise ImportError(f"{_LIB_PATH} is not built; run quantized_weight_exq_gb300/build.py "
                          "(or __graft_entry__.build())")
    lib = ctypes.CDLL(str(_LIB_PATH))
    P, i32, i64, sz, st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    W, dbl = ctypes.POINTER(exq_weight), ctypes.c_double
    sig = {
        "exq_pack_gptq": (st, [P, P, P, i32, i32, i32, P, P, P]),
        "exq_pack_exl2": (st, [P, P, i32, i32, P, P]),
        "exq_pack_exl2_qscale": (st, [P, i32, i32, P]),
        "exq_exl2_word_rows": (i64, [P, i32]),
        "exq_exl2_seg_word_off": (st, [P, i32, P]),
        "exq_dequant": (st, [W, P, P]),
        "exq_gemv_workspace_size": (sz, [W, i32]),
        "exq_gemv": (st, [W, P, i32, P, P, sz, P]),
        "exq_gemv_multi_workspace_size": (sz, [W, i32, i32]),
        "exq_gemv_multi": (st, [W, i32, P, i32, P, P, sz, P]),
        "exq_gemm_workspace_size": (sz, [W, i32]),
        "exq_gemm": (st, [W, P, i32, P, P, sz, P]),
        "exq_gemm_noalloc": (st, [W, P, i32, P, P]),
        "exq_gemm_multi_workspace_size": (sz, [W, i32, i32]),
        "exq_gemm_multi": (st, [W, i32, P, i32, P, P, sz, P]),
        "exq_kv_quantize": (st, [P, i64, i32, i32, P, P, P]),
        "exq_kv_dequantize": (st, [P, P, i64, i32, i32, P, P]),
        "exq_quantize_exl2": (st, [P, P, i32, i32, P, i32, P, P, P]),
        "exq_measure_exl2_workspace_size": (sz, [i32, i32]),
        "exq_measure_exl2": (st, [P, P, i32, i32, P, P, sz, P]),
        "exq_solve_exl2_bits": (st, [P, i32, i64, P]),
        "exq_rope_freqs": (st, [i32, dbl, i32, dbl, dbl, dbl, dbl, P, P]),
        "exq_rope_steps": (st, [P, i32, P]),
        "exq_rope": (st, [P, P, i64, i32, i32, P, P, i32, P]),
        "exq_kv_append": (st, [P, i32, P, P, P, P, P, P, P, i32, P]),
        "exq_paged_attn_workspace_size": (sz, [P, P, i32]),
        "exq_paged_attn": (st, [P, i32, P, P, i32, ctypes.c_float, i32, i32, P, P, P, sz, P]),
        "exq_kv_copy_pages": (st, [P, P, i64, P]),
        "exq_pages_alloc": (st, [P, i32, i32, P]),
        "exq_pages_free": (st, [P, i32, P, i32]),
        "exq_pages_fork": (st, [P, i32, i32, P, i32, P, P, P]),
        "exq_pages_compact": (st, [P, i32, P, i64, P, P]),
        "exq_fp4_scale_bytes": (sz, [i32, i32, i32]),
        "exq_pack_fp4": (st, [P, P, i32, i32, i32, P, P]),
        "exq_fp4_quantize": (st, [P, P, P]),
        "exq_fp4_dequantize": (st, [P, P, P]),
        "exq_fp4_gemm": (st, [P, P, P, P]),
        "exq_fp4_gemv_workspace_size": (sz, [P, i32]),
        "exq_fp4_gemv": (st, [P, P, i32, P, P, sz, P]),
        "exq_moe_workspace_size": (sz, [P, i32]),
        "exq_moe": (st, [P, P, i32, P, P, P, P, sz, P]),
        "exq_status_string": (ctypes.c_char_p, [st]),
        "exq_get_last_device_error": (st, [P]),
        "exq_testing_starve": (None, [i32]),
        "exq_testing_first_unit": (i64, [i32, i64, i32]),
        "exq_testing_unit_owner": (i32, [i64, i64, i32]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = _load()


def library_path() -> str:
    return str(_LIB_PATH)


def status_string(status: int) -> str:
    return _lib.exq_status_string(int(status)).decode()


exq_status_string = status_string


def _check(status: int, where: str):
    if status != EXQ_OK:
        raise ExqError(status, where)


def _np_ptr(a: Optional[np.ndarray]):
    return None if a is None else a.ctypes.data


def _stream_ptr(stream, device: Optional[int] = None) -> Optional[int]:
    """The handle of ``stream``, or of the current one (of ``device``, where the caller knows that it is the current device)."""
    if stream is None:
        import torch
        # the current stream's handle without the Stream object around it (3 us a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if device is None else device)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _on(stream, device):
    """The context in which ``stream`` (a torch stream, a handle, or None: the current one) is the current stream."""
    if stream is None:
        return contextlib.nullcontext()
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream_ptr(stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _empty(shape, dtype, device, stream):
    """Memory that a kernel launched on ``stream`` may write at once, and that the current stream may go on to use: of the
    allocator's pool for ``stream``, where what it held before was used in that stream's order."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    with _on(stream, device):
        t = torch.empty(shape, dtype=dtype, device=device)
        if torch.cuda.current_stream(device) != current:
            t.record_stream(current)
    return t


# ---------------------------------------------------------------- host packers

def exq_pack_gptq(q: np.ndarray, z: np.ndarray, g_idx: Optional[np.ndarray], group_size: int):
    """-> (qweight uint32 [K/8, N], qzeros uint32 [G, N/8], perm int32 [K])."""
    q = np.ascontiguousarray(q, dtype=np.uint8)
    z = np.ascontiguousarray(z, dtype=np.uint8)
    K, N = q.shape
    gi = None if g_idx is None else np.ascontiguousarray(g_idx, dtype=np.int32)
    qweight = np.empty((K // 8, N), dtype=np.uint32)
    qzeros = np.empty((max(K // max(group_size, 1), 1), N // 8), dtype=np.uint32)
    perm = np.empty(K, dtype=np.int32)
    _check(_lib.exq_pack_gptq(_np_ptr(q), _np_ptr(z), _np_ptr(gi), K, N, group_size,
                              _np_ptr(qweight), _np_ptr(qzeros), _np_ptr(perm)), "exq_pack_gptq")
    return qweight, qzeros, perm


def exq_exl2_word_rows(bits: np.ndarray) -> int:
    bits = np.ascontiguousarray(bits, dtype=np.uint8)
    return int(_lib.exq_exl2_word_rows(_np_ptr(bits), bits.size))


def exq_exl2_seg_word_off(bits: np.ndarray) -> np.ndarray:
    """Segment table uint32 [S + 1] (word-row prefix sums) of the widths [S]."""
    bits = np.ascontiguousarray(bits, dtype=np.uint8)
    off = np.empty(bits.size + 1, dtype=np.uint32)
    _check(_lib.exq_exl2_seg_word_off(_np_ptr(bits), bits.size, _np_ptr(off)), "exq_exl2_seg_word_off")
    return off


def exq_pack_exl2(q: np.ndarray, bits: np.ndarray):
    """-> (qweight uint32 [sum(bits), N], seg_word_off uint32 [S + 1])."""
    q = np.ascontiguousarray(q, dtype=np.uint8)
    bits = np.ascontiguousarray(bits, dtype=np.uint8)
    K, N = q.shape
    rows = exq_exl2_word_rows(bits)
    if rows < 0:
        raise ExqError(EXQ_ERR_INVALID_ARG, "exq_pack_exl2")
    qweight = np.empty((rows, N), dtype=np.uint32)
    off = np.empty(bits.size + 1, dtype=np.uint32)
    _check(_lib.exq_pack_exl2(_np_ptr(q), _np_ptr(bits), K, N, _np_ptr(qweight), _np_ptr(off)), "exq_pack_exl2")
    return qweight, off


def exq_pack_exl2_qscale(codes: np.ndarray) -> np.ndarray:
    """4-bit scale codes uint8 [S, N] -> q_scale uint32 [S, N/8]."""
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    S, N = codes.shape
    out = np.empty((S, max(N // 8, 1)), dtype=np.uint32)
    _check(_lib.exq_pack_exl2_qscale(_np_ptr(codes), S, N, _np_ptr(out)), "exq_pack_exl2_qscale")
    return out


# ---------------------------------------------------------------- device layer

@dataclass
class Weight:
    """A packed layer resident on the GPU (torch tensors hold the memory)."""

    format: int
    K: int
    N: int
    group_size: int
    qweight: "object"                 # torch.int32 [rows, N] (uint32 bits)
    scales: "object"                  # torch.float16 [G or S, N]; None for EXL2 two-level
    qzeros: "object" = None           # torch.int32 [G, N/8] (GPTQ)
    perm: "object" = None             # torch.int32 [K]
    seg_word_off: "object" = None     # torch.int32 [S + 1] (EXL2)
    q_scale: "object" = None          # torch.int32 [S, N/8] 4-bit codes (EXL2 two-level)
    q_scale_max: "object" = None      # torch.float16 [N] (EXL2 two-level)
    _desc: exq_weight = field(default=None, repr=False)

    def desc(self) -> exq_weight:
        if self._desc is None:
            ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
            groups = self.scales.shape[0] if self.scales is not None else self.q_scale.shape[0]
            self._desc = exq_weight(
                self.format, self.K, self.N, self.group_size, groups, self.qweight.shape[0],
                ptr(self.qweight), ptr(self.scales), ptr(self.qzeros), ptr(self.perm), ptr(self.seg_word_off),
                ptr(self.q_scale), ptr(self.q_scale_max))
        return self._desc

    @property
    def packed_bytes(self) -> int:
        """qweight + scales (or scale codes and column maxima) + qzeros bytes:
        the weight stream of one matmul."""
        n = self.qweight.numel() * 4
        for t, size in ((self.scales, 2), (self.qzeros, 4), (self.q_scale, 4), (self.q_scale_max, 2)):
            if t is not None:
                n += t.numel() * size
        return n


def _dev(a, dtype, device):
    import torch
    if a is None:
        return None
    if isinstance(a, torch.Tensor):
        return a.to(device=device).contiguous()
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint32:
        a = a.view(np.int32)
    if a.dtype == np.uint16:
        a = a.view(np.float16)
    return torch.from_numpy(a).to(device=device, dtype=dtype).contiguous()


def gptq_weight(qweight, qzeros, scales, perm, K: int, N: int, group_size: int, device="cuda") -> Weight:
    import torch
    return Weight(EXQ_FMT_GPTQ4, K, N, group_size, _dev(qweight, torch.int32, device),
                  _dev(scales, torch.float16, device), _dev(qzeros, torch.int32, device),
                  _dev(perm, torch.int32, device), None)


def exl2_weight(qweight, seg_word_off, scales, perm, K: int, N: int, device="cuda") -> Weight:
    import torch
    return Weight(EXQ_FMT_EXL2, K, N, 32, _dev(qweight, torch.int32, device),
                  _dev(scales, torch.float16, device), None, _dev(perm, torch.int32, device),
                  _dev(seg_word_off, torch.int32, device))


def exl2_qscale_weight(qweight, seg_word_off, q_scale, q_scale_max, perm, K: int, N: int, device="cuda") -> Weight:
    """EXL2 layer with two-level scales: q_scale uint32 [S, N/8] packed codes
    (exq_pack_exl2_qscale), q_scale_max fp16 [N]."""
    import torch
    return Weight(EXQ_FMT_EXL2_QSCALE, K, N, 32, _dev(qweight, torch.int32, device), None, None,
                  _dev(perm, torch.int32, device), _dev(seg_word_off, torch.int32, device),
                  _dev(q_scale, torch.int32, device), _dev(q_scale_max, torch.float16, device))


def exq_dequant(w: Weight, W_out, stream=None):
    _check(_lib.exq_dequant(ctypes.byref(w.desc()), W_out.data_ptr(), _stream_ptr(stream)), "exq_dequant")
    return W_out


def exq_gemv_workspace_size(w: Weight, M: int) -> int:
    return int(_lib.exq_gemv_workspace_size(ctypes.byref(w.desc()), M))


_gemv_ws = {}       # device index -> zero-filled uint8 workspace shared by calls on one stream
_gemv_ws_outgrown = []  # smaller ones from before: graphs captured with them keep their addresses


def gemv_workspace(w: Weight, M: int):
    """A zero-filled exq_gemv workspace for the current device, kept and grown
    across calls. exq_gemv leaves it zeroed, so calls ordered on one stream can
    share it; calls that may overlap on the GPU need their own (torch.zeros of
    exq_gemv_workspace_size bytes)."""
    return _shared_workspace(exq_gemv_workspace_size(w, M))


def _shared_workspace(need: int):
    import torch
    dev = torch.cuda.current_device()
    buf = _gemv_ws.get(dev)
    if buf is None or buf.numel() < need:
        if buf is not None:
            _gemv_ws_outgrown.append(buf)
        buf = torch.zeros(max(need, 1 << 20, 2 * buf.numel() if buf is not None else 0), dtype=torch.uint8, device=f"cuda:{dev}")
        _gemv_ws[dev] = buf
    return buf


_attn_ws = {}  # (device index, stream handle) -> zero-filled uint8 workspace of exq_paged_attn


def _attn_workspace(need: int, dev: int, stream, handle: int):
    """The default exq_paged_attn workspace of the launch's stream, zeroed in that stream's order; kept and grown across calls.
    Refused while the stream is captured: a graph needs a workspace that lives as long as it does."""
    import torch
    if stream is not None:
        with _on(stream, dev):
            return _attn_workspace(need, dev, None, handle)
    if torch.cuda.is_current_stream_capturing():
        raise ExqError(EXQ_ERR_INVALID_ARG, "exq_paged_attn")
    buf = _attn_ws.get((dev, handle))
    if buf is None or buf.numel() < need:
        # (the outgrown one goes back to the stream's own pool: what runs on the stream still has it)
        buf = _attn_ws[dev, handle] = torch.zeros(max(need, 1 << 20), dtype=torch.uint8, device=f"cuda:{dev}")
    return buf


def exq_gemv(w: Weight, x, y, workspace=None, stream=None):
    if workspace is None:
        workspace = gemv_workspace(w, x.shape[0])
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(_lib.exq_gemv(ctypes.byref(w.desc()), x.data_ptr(), x.shape[0], y.data_ptr(), workspace.data_ptr(),
                         ws_bytes, _stream_ptr(stream)), "exq_gemv")
    return y


def _desc_array(ws):
    return (exq_weight * len(ws))(*[w.desc() for w in ws])


def exq_gemv_multi_workspace_size(ws, M: int) -> int:
    return int(_lib.exq_gemv_multi_workspace_size(_desc_array(ws), len(ws), M))


def exq_gemv_multi(ws, x, ys, workspace=None, stream=None):
    """y_i = x . dequant(ws[i]) for the layers ws (one format, one K), in one
    launch. ``ys`` are the outputs, one per layer."""
    if len(ws) != len(ys):
        raise ExqError(EXQ_ERR_INVALID_ARG, "exq_gemv_multi")
    if workspace is None:
        workspace = _shared_workspace(exq_gemv_multi_workspace_size(ws, x.shape[0]))
    ws_bytes = workspace.numel() * workspace.element_size()
    yp = (ctypes.c_void_p * len(ys))(*[y.data_ptr() for y in ys])
    _check(_lib.exq_gemv_multi(_desc_array(ws), len(ws), x.data_ptr(), x.shape[0], yp, workspace.data_ptr(),
                               ws_bytes, _stream_ptr(stream)), "exq_gemv_multi")
    return ys


def exq_gemm_workspace_size(w: Weight, M: int) -> int:
    return int(_lib.exq_gemm_workspace_size(ctypes.byref(w.desc()), M))


def exq_gemm(w: Weight, x, y, workspace=None, stream=None):
    ws_ptr = None if workspace is None else workspace.data_ptr()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.exq_gemm(ctypes.byref(w.desc()), x.data_ptr(), x.shape[0], y.data_ptr(), ws_ptr, ws_bytes,
                         _stream_ptr(stream)), "exq_gemm")
    return y


def exq_gemm_multi_workspace_size(ws, M: int) -> int:
    return int(_lib.exq_gemm_multi_workspace_size(_desc_array(ws), len(ws), M))


def exq_gemm_multi(ws, x, ys, workspace=None, stream=None):
    """y_i = x . dequant(ws[i]) for the layers ws (one format, one K), in one
    prefill launch. ``ys`` are the outputs, one per layer."""
    import torch
    if len(ws) != len(ys):
        raise ExqError(EXQ_ERR_INVALID_ARG, "exq_gemm_multi")
    need = exq_gemm_multi_workspace_size(ws, x.shape[0])
    if workspace is None and need:
        workspace = _empty(need, torch.uint8, x.device, stream)
    ws_ptr = None if workspace is None else workspace.data_ptr()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    yp = (ctypes.c_void_p * len(ys))(*[y.data_ptr() for y in ys])
    _check(_lib.exq_gemm_multi(_desc_array(ws), len(ws), x.data_ptr(), x.shape[0], yp, ws_ptr, ws_bytes,
                               _stream_ptr(stream)), "exq_gemm_multi")
    return ys


GEMM_MAX_LAYERS = 4


def exq_gemm_noalloc(w: Weight, x, y, stream=None):
    """exq_gemm for callers that cannot allocate: an act-order layer's
    gathered activations go to the library's static scratch array (see
    include/exq.h for the size limit, the first-call set-up and the rule that
    overlapping calls race on the shared array)."""
    _check(_lib.exq_gemm_noalloc(ctypes.byref(w.desc()), x.data_ptr(), x.shape[0], y.data_ptr(),
                                 _stream_ptr(stream)), "exq_gemm_noalloc")
    return y


def exq_kv_quantize(x, bits: int, codes=None, scales=None, stream=None):
    """Quantized KV cache write: x fp16 [..., D] (groups of D values) ->
    (codes int32 [groups, D * bits / 32] holding uint32 words, scales fp16 [groups])."""
    import torch
    D = x.shape[-1]
    G = x.numel() // D if D else 0
    if codes is None:
        codes = _empty((G, D * bits // 32), torch.int32, x.device, stream)
    if scales is None:
        scales = _empty(G, torch.float16, x.device, stream)
    _check(_lib.exq_kv_quantize(x.data_ptr(), G, D, bits, codes.data_ptr(), scales.data_ptr(), _stream_ptr(stream)),
           "exq_kv_quantize")
    return codes, scales


def exq_kv_dequantize(codes, scales, D: int, bits: int, out=None, stream=None):
    """Quantized KV cache read: fp16 [groups, D]."""
    import torch
    G = scales.numel()
    if out is None:
        out = _empty((G, D), torch.float16, scales.device, stream)
    _check(_lib.exq_kv_dequantize(codes.data_ptr(), scales.data_ptr(), G, D, bits, out.data_ptr(),
                                  _stream_ptr(stream)), "exq_kv_dequantize")
    return out


# ---------------------------------------------------------------- rotary positions

def _here(where: str, *devices: int) -> None:
    """Refuses tensors (their get_device()) of different devices, of the host, or of another device than the current one,
    which the launch goes to: its kernels could not read them."""
    import torch
    d = devices[0]
    if d < 0 or devices.count(d) != len(devices) or d != torch.cuda.current_device():
        raise ExqError(EXQ_ERR_INVALID_ARG, where)


def exq_rope_freqs(R: int, base: float = 10000.0, scaling: int = ROPE_SCALE_NONE, factor: float = 1.0,
                   orig_ctx: float = 0.0, low: float = 1.0, high: float = 32.0):
    """Host: (frequencies float64 [R/2] in radians per position, gain)."""
    out = np.empty(max(int(R) // 2, 1), dtype=np.float64)
    gain = ctypes.c_double()
    _check(_lib.exq_rope_freqs(R, base, scaling, factor, orig_ctx, low, high, _np_ptr(out), ctypes.byref(gain)),
           "exq_rope_freqs")
    return out, gain.value


def exq_rope_steps(inv_freq: np.ndarray) -> np.ndarray:
    """Host: frequencies (radians per position) -> uint64 turns per position in units of 2^-64."""
    f = np.ascontiguousarray(inv_freq, dtype=np.float64)
    out = np.empty(f.size, dtype=np.uint64)
    _check(_lib.exq_rope_steps(_np_ptr(f), f.size, _np_ptr(out)), "exq_rope_steps")
    return out


class Rope:
    """Rotary parameters on the GPU: steps int64 [R/2] (uint64 bits, exq_rope_steps), the layout and the gain."""

    def __init__(self, steps, R: int, layout: int = ROPE_HALF, gain: float = 1.0):
        if (not steps.is_cuda or steps.numel() < R // 2 or steps.element_size() != 8 or steps.is_floating_point()
                or not steps.is_contiguous()):
            raise ExqError(EXQ_ERR_INVALID_ARG, "Rope")
        self.steps, self.R, self.layout, self.gain = steps, R, layout, gain
        self._desc = exq_rope_params(steps.data_ptr(), R, layout, gain)


def rope_table(R: int, layout: int = ROPE_HALF, device="cuda", **freqs) -> Rope:
    """A Rope from exq_rope_freqs(R, **freqs) and exq_rope_steps."""
    import torch
    f, gain = exq_rope_freqs(R, **freqs)
    return Rope(torch.from_numpy(exq_rope_steps(f).view(np.int64)).to(device), R, layout, gain)


def _rows(x, where: str, D: Optional[int] = None, heads: Optional[int] = None, tokens: Optional[int] = None):
    """Descriptor of fp16 [tokens, heads, D] with a contiguous last axis, on the device that _here has seen."""
    import torch
    t, h, d = x.shape
    st, sh, sd = x.stride()
    if (x.dtype != torch.float16 or (sd != 1 and d > 1) or (D is not None and d != D)
            or (heads is not None and h != heads) or (tokens is not None and t < tokens)):
        raise ExqError(EXQ_ERR_INVALID_ARG, where)
    return exq_rows(x.data_ptr(), st, sh)


def exq_rope(x, pos, rope: Rope, out=None, grad: bool = False, stream=None):
    """x fp16 [tokens, heads, D] turned by the positions pos int32 [tokens] (grad: the transposed map, from the gradient at
    the result to the gradient at x). ``out`` may be x."""
    import torch
    T, H, D = x.shape
    if not pos.is_cuda or pos.numel() < T or pos.dtype != torch.int32 or not pos.is_contiguous():
        raise ExqError(EXQ_ERR_INVALID_ARG, "exq_rope")
    dev = x.get_device()
    _here("exq_rope", dev, pos.get_device(), rope.steps.get_device(), dev if out is None else out.get_device())
    if out is None:
        out = _empty((T, H, D), torch.float16, x.device, stream)
    xr, yr = _rows(x, "exq_rope"), _rows(out, "exq_rope", D, H, T)
    _check(_lib.exq_rope(ctypes.byref(rope._desc), ctypes.byref(xr), T, H, D, pos.data_ptr(), ctypes.byref(yr), int(grad),
                         _stream_ptr(stream, dev)), "exq_rope")
    return out


# ---------------------------------------------------------------- paged KV cache

class KVCache:
    """A paged cache on the GPU: k_codes, v_codes int32 [layers, pages, KV heads, page_size, D * bits / 32] (uint32 words;
    fp16 pairs for bits 16), k_scales, v_scales fp16 [layers, pages, KV heads, page_size] (None for bits 16)."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales, bits: int):
        import torch
        shape = k_codes.shape
        L, P, H, S, W = shape
        quantised = bits != 16
        self.device = dev = k_codes.get_device()
        if (dev < 0 or v_codes.get_device() != dev or k_codes.dtype != torch.int32 or v_codes.dtype != torch.int32
                or v_codes.shape != shape or W * 32 % bits
                or not k_codes.is_contiguous() or not v_codes.is_contiguous()
                or (k_scales is not None) != quantised or (v_scales is not None) != quantised):
            raise ExqError(EXQ_ERR_INVALID_ARG, "KVCache")
        if quantised and (k_scales.get_device() != dev or v_scales.get_device() != dev
                          or k_scales.dtype != torch.float16 or v_scales.dtype != torch.float16
                          or k_scales.shape != shape[:4] or v_scales.shape != shape[:4]
                          or not k_scales.is_contiguous() or not v_scales.is_contiguous()):
            raise ExqError(EXQ_ERR_INVALID_ARG, "KVCache")
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.bits, self.D, self.n_kv_heads, self.page_size, self.n_pages, self.n_layers = bits, W * 32 // bits, H, S, P, L
        self._desc = exq_kv_cache(bits, self.D, H, S, P, L, k_codes.data_ptr(),
                                  None if k_scales is None else k_scales.data_ptr(), v_codes.data_ptr(),
                                  None if v_scales is None else v_scales.data_ptr())


def kv_cache(n_layers: int, n_pages: int, n_kv_heads: int, page_size: int, D: int, bits: int, device="cuda") -> KVCache:
    """A KVCache with memory of its own (contents undefined until exq_kv_append writes them)."""
    import torch
    shape = (n_layers, n_pages, n_kv_heads, page_size)
    codes = [torch.empty(*shape, D * bits // 32, dtype=torch.int32, device=device) for _ in range(2)]
    scales = [None if bits == 16 else torch.empty(shape, dtype=torch.float16, device=device) for _ in range(2)]
    return KVCache(*codes, *scales, bits)


class KVBatch:
    """The sequences of one step: q_start int32 [B + 1], kv_len int32 [B], page_table int32 [B, max_pages] on the GPU, and
    the host's bounds on new and cached tokens of any sequence (see exq_kv_batch). n_tokens: rows of q, k and v."""

    def __init__(self, q_start, kv_len, page_table, max_q_len: int, max_kv_len: int, n_tokens: Optional[int] = None):
        B, pages = page_table.shape
        import torch
        i32 = torch.int32
        self.device = dev = q_start.get_device()
        if (dev < 0 or kv_len.get_device() != dev or page_table.get_device() != dev or q_start.dtype != i32
                or kv_len.dtype != i32 or page_table.dtype != i32 or q_start.shape != (B + 1,)
                or kv_len.shape != (B,) or not q_start.is_contiguous() or not kv_len.is_contiguous()
                or not page_table.is_contiguous()):
            raise ExqError(EXQ_ERR_INVALID_ARG, "KVBatch")
        self.q_start, self.kv_len, self.page_table, self.n_tokens = q_start, kv_len, page_table, n_tokens
        self._rest = max_q_len, max_kv_len, pages, q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr()
        self._last = -1, None

    def desc(self, rows: int) -> exq_kv_batch:
        """The descriptor of a call with ``rows`` rows. One that has been handed out is not written again: another thread's
        call with the same batch may have other rows."""
        if self.n_tokens is not None:
            rows = self.n_tokens
        last, d = self._last
        if last != rows:
            d = exq_kv_batch(self.kv_len.shape[0], rows, *self._rest)
            self._last = rows, d
        return d


def exq_kv_append(cache: KVCache, batch: KVBatch, k, v, q=None, rope: Optional[Rope] = None, pos=None, q_out=None,
                  layer: int = 0, stream=None):
    """Writes the new tokens' k and v, fp16 [tokens, KV heads, D], to their slots of one layer, k (and q, fp16 [tokens,
    heads, D], where given) turned by ``rope``. Returns the turned q (``q_out``, which may be q) or None."""
    import torch
    where = "exq_kv_append"
    T, H, D = k.shape[0], cache.n_kv_heads, cache.D
    if batch.n_tokens is not None:
        if batch.n_tokens > T:
            raise ExqError(EXQ_ERR_INVALID_ARG, where)
        T = batch.n_tokens
    dev = cache.device
    _here(where, dev, batch.device, k.get_device(), v.get_device(), dev if q is None else q.get_device(),
          dev if q_out is None else q_out.get_device(), dev if pos is None else pos.get_device(),
          dev if rope is None else rope.steps.get_device())
    kr, vr = _rows(k, where, D, H), _rows(v, where, D, H, T)
    qp = op = None
    heads = 0
    if q is not None:
        heads = q.shape[1]
        if q_out is None:
            q_out = _empty(q.shape, torch.float16, q.device, stream)
        qp, op = ctypes.byref(_rows(q, where, D, None, T)), ctypes.byref(_rows(q_out, where, D, heads, T))
    if pos is not None and (pos.numel() < T or pos.dtype != torch.int32 or not pos.is_contiguous()):
        raise ExqError(EXQ_ERR_INVALID_ARG, where)
    _check(_lib.exq_kv_append(ctypes.byref(cache._desc), layer, ctypes.byref(batch.desc(T)), ctypes.byref(kr),
                              ctypes.byref(vr), None if rope is None else ctypes.byref(rope._desc),
                              None if pos is None else pos.data_ptr(), qp, op, heads, _stream_ptr(stream, dev)), where)
    return q_out if q is not None else None


def exq_paged_attn_workspace_size(cache: KVCache, batch: KVBatch, n_heads: int, n_tokens: int) -> int:
    return int(_lib.exq_paged_attn_workspace_size(ctypes.byref(cache._desc), ctypes.byref(batch.desc(n_tokens)), n_heads))


def exq_paged_attn(cache: KVCache, batch: KVBatch, q, out=None, scale: Optional[float] = None, causal: bool = True,
                   window: int = 0, lse=None, layer: int = 0, workspace=None, stream=None):
    """Attention of the new tokens' q, fp16 [tokens, heads, D], over the cached tokens of their sequences, the new ones
    among them (exq_kv_append first). scale: 1 / sqrt(D) unless given; lse: fp32 [tokens, heads] to fill, or None.
    Without ``workspace`` one is kept for each stream that calls are launched on. A call that a graph captures needs one
    of its own, for as long as the graph is replayed."""
    import torch
    where = "exq_paged_attn"
    T, H, D = q.shape
    if batch.n_tokens is not None:
        if batch.n_tokens > T:
            raise ExqError(EXQ_ERR_INVALID_ARG, where)
        T = batch.n_tokens
    dev = cache.device
    _here(where, dev, batch.device, q.get_device(), dev if out is None else out.get_device(),
          dev if lse is None else lse.get_device(), dev if workspace is None else workspace.get_device())
    if out is None:
        out = _empty(q.shape, torch.float16, q.device, stream)
    qr, orow = _rows(q, where, cache.D), _rows(out, where, cache.D, H, T)
    if lse is not None and (lse.dtype != torch.float32 or lse.numel() < T * H or not lse.is_contiguous()):
        raise ExqError(EXQ_ERR_INVALID_ARG, where)
    c, b, handle = ctypes.byref(cache._desc), ctypes.byref(batch.desc(T)), _stream_ptr(stream, dev)
    if workspace is None:
        workspace = _attn_workspace(int(_lib.exq_paged_attn_workspace_size(c, b, H)), dev, stream, handle)
    _check(_lib.exq_paged_attn(c, layer, b, ctypes.byref(qr), H, D ** -0.5 if scale is None else scale, int(causal), window,
                               ctypes.byref(orow), None if lse is None else lse.data_ptr(), workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), handle), where)
    return out


def exq_kv_copy_pages(cache: KVCache, pairs, stream=None) -> None:
    """Copies pages pairs int32 [n, 2] of (src, dst) on the GPU, in every layer."""
    import torch
    if not pairs.is_cuda or pairs.dtype != torch.int32 or not pairs.is_contiguous() or pairs.numel() % 2:
        raise ExqError(EXQ_ERR_INVALID_ARG, "exq_kv_copy_pages")
    _here("exq_kv_copy_pages", cache.device, pairs.get_device())
    _check(_lib.exq_kv_copy_pages(ctypes.byref(cache._desc), pairs.data_ptr(), pairs.numel() // 2,
                                  _stream_ptr(stream, cache.device)),
           "exq_kv_copy_pages")


# ---------------------------------------------------------------- microscaled 4-bit floating point

FP4_COUNTER_BYTES = 128 << 10  # EXQ_FP4_COUNTER_BYTES

# (device index, stream handle) -> (workspace of exq_fp4_gemv and exq_moe, its address and bytes); its counters are zero between calls
_fp4_ws = {}
_fp4_locks = {}


def _fp4_lock(dev: int, handle: int):
    """Held by the host thread that has the default workspace of a stream, from before it is looked up until the call's launches
    are all made: they pass data through it, and another thread's may not come between them, nor another workspace be put in its place."""
    return _fp4_locks.get((dev, handle)) or _fp4_locks.setdefault((dev, handle), threading.RLock())


def _fp4_workspace(need: int, dev: int, stream, handle: int, where: str):
    """(memory, address, bytes) of the default workspace of the launch's stream, its counters zeroed in that stream's order; kept and
    grown across calls, under _fp4_lock. Refused while the stream is captured: a graph needs a workspace that lives as long as it does."""
    import torch
    if stream is not None:
        with _on(stream, dev):
            return _fp4_workspace(need, dev, None, handle, where)
    if torch.cuda.is_current_stream_capturing():
        raise ExqError(EXQ_ERR_INVALID_ARG, where)
    kept = _fp4_ws.get((dev, handle))
    if kept is None or kept[2] < need:
        buf = torch.empty(max(need, 8 << 20), dtype=torch.uint8, device=f"cuda:{dev}")
        buf[:FP4_COUNTER_BYTES].zero_()
        kept = _fp4_ws[dev, handle] = buf, buf.data_ptr(), buf.numel()
    return kept


def exq_fp4_scale_bytes(format: int, rows: int, K: int) -> int:
    return int(_lib.exq_fp4_scale_bytes(format, rows, K))


def _fp4_tensors(where: str, codes, scales, lead: tuple, format: int):
    """(rows, K) of codes uint8 [*lead, rows, K / 2] with scales uint8 [*lead, bytes], both contiguous and on one device."""
    import torch
    if (codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or codes.dim() != len(lead) + 2 or codes.get_device() < 0
            or scales.get_device() != codes.get_device() or not codes.is_contiguous() or not scales.is_contiguous()):
        raise ExqError(EXQ_ERR_INVALID_ARG, where)
    rows, K = codes.shape[-2], 2 * codes.shape[-1]
    if codes.shape[:-2] != lead or (rows and tuple(scales.shape) != (*lead, exq_fp4_scale_bytes(format, rows, K))):
        raise ExqError(EXQ_ERR_INVALID_ARG, where)
    return rows, K


class Fp4Matrix:
    """A matrix [rows, K] in the 4-bit format on the GPU: codes uint8 [rows, K / 2], scales uint8 [exq_fp4_scale_bytes] in tiles
    (exq_pack_fp4, exq_fp4_quantize), and the factor of an E4M3 one, a float of 64 bits as the caller gave it (the quantiser decides
    with it; where values are multiplied by it, it is rounded to 32 bits)."""

    __slots__ = "rows", "K", "format", "factor", "device", "_buf", "_codes", "_scales", "_desc", "_ref", "_space"

    def __init__(self, codes, scales, format: int, factor: float = 1.0):
        self.rows, self.K = _fp4_tensors("Fp4Matrix", codes, scales, (), format)
        self._buf, self._codes, self._scales, self.format, self.factor = None, codes, scales, format, factor
        self._space = {}
        self.device = codes.get_device()
        self._desc = exq_fp4_matrix(format, self.rows, self.K, factor, codes.data_ptr(), scales.data_ptr())
        self._ref = ctypes.byref(self._desc)

    @classmethod
    def _made(cls, rows: int, K: int, format: int, factor: float, like, stream):
        """One with memory of its own (codes, then scales), on the device of ``like``; its sizes are for the call that fills it to check."""
        import torch
        m = cls.__new__(cls)
        n = rows * K // 2
        size = n + 512 * (-(-rows // 128) * -(-K // (64 if format == FP4_E4M3 else 128)))
        m._buf = buf = (torch.empty(size, dtype=torch.uint8, device=like.device) if stream is None
                        else _empty(size, torch.uint8, like.device, stream))
        m.rows, m.K, m.format, m.factor, m.device = rows, K, format, factor, like.get_device()
        m._codes = m._scales = m._space = None
        at = buf.data_ptr()
        m._desc = d = exq_fp4_matrix(format, rows, K, factor, at, at + n)
        m._ref = ctypes.byref(d)
        return m

    @property
    def codes(self):
        if self._codes is None:
            self._codes = self._buf[:self.rows * self.K // 2].view(self.rows, self.K // 2)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self._scales = self._buf[self.rows * self.K // 2:]
        return self._scales


def exq_pack_fp4(codes: np.ndarray, scales: np.ndarray, format: int):
    """Host: codes uint8 [rows, K] (0..15) and scale bytes uint8 [rows, K / block] -> (codes uint8 [rows, K / 2], scales uint8
    [exq_fp4_scale_bytes]) as the matrices of the library have them."""
    codes, scales = np.ascontiguousarray(codes, dtype=np.uint8), np.ascontiguousarray(scales, dtype=np.uint8)
    rows, K = codes.shape
    if format not in (FP4_E4M3, FP4_E8M0) or scales.shape != (rows, K // (16 if format == FP4_E4M3 else 32)):
        raise ExqError(EXQ_ERR_INVALID_ARG, "exq_pack_fp4")
    out, tiles = np.empty((rows, K // 2), np.uint8), np.empty(exq_fp4_scale_bytes(format, rows, K), np.uint8)
    _check(_lib.exq_pack_fp4(_np_ptr(codes), _np_ptr(scales), format, rows, K, _np_ptr(out), _np_ptr(tiles)), "exq_pack_fp4")
    return out, tiles


def fp4_matrix(codes: np.ndarray, scales: np.ndarray, format: int, factor: float = 1.0, device="cuda") -> Fp4Matrix:
    """An Fp4Matrix of host codes [rows, K] and scale bytes [rows, K / block]."""
    import torch
    return Fp4Matrix(*(torch.from_numpy(a).to(device) for a in exq_pack_fp4(codes, scales, format)), format, factor)


def _is_rows(x, half) -> bool:
    return x.dtype is half and x.dim() == 2 and x.is_contiguous()


def _result(out, rows: int, cols: int, dev: int, like, stream, where: str):
    """``out``, which has to be a contiguous fp16 [rows, cols] on the device, or such a tensor."""
    import torch
    if out is None:
        if stream is None:
            return torch.empty((rows, cols), dtype=torch.float16, device=like.device)
        return _empty((rows, cols), torch.float16, like.device, stream)
    if not _is_rows(out, torch.float16) or out.shape != (rows, cols) or out.get_device() != dev:
        raise ExqError(EXQ_ERR_INVALID_ARG, where)
    return out


def exq_fp4_quantize(x, format: int, factor: float = 1.0, out: Optional[Fp4Matrix] = None, stream=None) -> Fp4Matrix:
    """x fp16 [rows, K] in the 4-bit format: a new Fp4Matrix, or ``out`` (whose format and factor are taken) with its contents
    replaced."""
    import torch
    where = "exq_fp4_quantize"
    dev = x.get_device()
    _here(where, dev)
    if not _is_rows(x, torch.float16):
        raise ExqError(EXQ_ERR_INVALID_ARG, where)
    rows, K = x.shape
    if out is None:
        out = Fp4Matrix._made(rows, K, format, factor, x, stream)
    elif out.rows != rows or out.K != K or out.device != dev:
        raise ExqError(EXQ_ERR_INVALID_ARG, where)
    _check(_lib.exq_fp4_quantize(x.data_ptr(), out._ref, _stream_ptr(stream, dev)), where)
    return out


def exq_fp4_dequantize(m: Fp4Matrix, out=None, stream=None):
    """The matrix as fp16 [rows, K]."""
    where = "exq_fp4_dequantize"
    dev = m.device
    _here(where, dev)
    out = _result(out, m.rows, m.K, dev, m._codes if m._codes is not None else m._buf, stream, where)
    _check(_lib.exq_fp4_dequantize(m._ref, out.data_ptr(), _stream_ptr(stream, dev)), where)
    return out


def _space(workspace, dev: int, where: str):
    """(address, bytes) of a caller's workspace."""
    if not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ExqError(EXQ_ERR_INVALID_ARG, where)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def exq_fp4_gemm(a: Fp4Matrix, w: Fp4Matrix, out=None, stream=None):
    """a . w^T as fp16 [a.rows, w.rows], both in the 4-bit format."""
    where = "exq_fp4_gemm"
    dev = a.device
    _here(where, dev, w.device)
    out = _result(out, a.rows, w.rows, dev, a._codes if a._codes is not None else a._buf, stream, where)
    _check(_lib.exq_fp4_gemm(a._ref, w._ref, out.data_ptr(), _stream_ptr(stream, dev)), where)
    return out


def exq_fp4_gemv_workspace_size(w: Fp4Matrix, M: int) -> int:
    return int(_lib.exq_fp4_gemv_workspace_size(w._ref, M))


def exq_fp4_gemv(w: Fp4Matrix, x, out=None, workspace=None, stream=None):
    """x . w^T as fp16 [M, w.rows] for up to 16 rows x fp16 [M, K], which are not quantised. Without ``workspace`` one is kept for
    each stream that calls are launched on (calls of several host threads on one stream take turns). One that is given is for one
    call at a time: threads that share it take turns themselves. A call that a graph captures needs one of its own, its first FP4_COUNTER_BYTES zero,
    for as long as the graph is replayed."""
    import torch
    where = "exq_fp4_gemv"
    dev = w.device
    _here(where, dev, x.get_device())
    if not _is_rows(x, torch.float16) or x.shape[1] != w.K:
        raise ExqError(EXQ_ERR_INVALID_ARG, where)
    M = x.shape[0]
    out = _result(out, M, w.rows, dev, x, stream, where)
    handle = _stream_ptr(stream, dev)
    if workspace is None:
        if w._space is None:
            w._space = {}
        need = w._space.get(M)  # what M rows need, of a matrix of this shape
        if need is None:
            need = w._space[M] = _lib.exq_fp4_gemv_workspace_size(w._ref, M)
        with _fp4_lock(dev, handle):
            _kept, ws, n = _fp4_workspace(need, dev, stream, handle, where)
            status = _lib.exq_fp4_gemv(w._ref, x.data_ptr(), M, out.data_ptr(), ws, n, handle)
    else:
        ws, n = _space(workspace, dev, where)
        status = _lib.exq_fp4_gemv(w._ref, x.data_ptr(), M, out.data_ptr(), ws, n, handle)
    _check(status, where)
    return out


# ---------------------------------------------------------------- mixture of experts

class Fp4Experts:
    """One matrix [rows, K] for each expert, in the 4-bit format on the GPU: codes uint8 [experts, rows, K / 2], scales uint8
    [experts, exq_fp4_scale_bytes], factors fp32 [experts] (E4M3) or None."""

    def __init__(self, codes, scales, format: int, factors=None):
        import torch
        where = "Fp4Experts"
        self.rows, self.K = _fp4_tensors(where, codes, scales, (codes.shape[0],), format)
        self.n_experts, self.device = codes.shape[0], codes.get_device()
        if factors is not None and (factors.dtype != torch.float32 or factors.shape != (self.n_experts,)
                                    or factors.get_device() != self.device or not factors.is_contiguous()):
            raise ExqError(EXQ_ERR_INVALID_ARG, where)
        self.codes, self.scales, self.format, self.factors = codes, scales, format, factors
        self._desc = exq_fp4_experts(format, self.n_experts, self.rows, self.K, codes.data_ptr(), scales.data_ptr(),
                                     None if factors is None else factors.data_ptr())


class MoeLayer:
    """A layer of experts: gate and up [I, D], down [D, I] of each, the router fp16 [experts, D] (None: the calls bring ids and
    weights), how many experts a token has, and whether their weights add up to one."""

    def __init__(self, gate: Fp4Experts, up: Fp4Experts, down: Fp4Experts, top_k: int, router=None, renorm: bool = True,
                 act: int = ACT_SILU):
        import torch
        self.device, self.D, self.top_k = gate.device, gate.K, top_k
        if (up.device != self.device or down.device != self.device or
                (router is not None and (router.dtype != torch.float16 or router.shape != (gate.n_experts, gate.K)
                                         or router.get_device() != self.device or not router.is_contiguous()))):
            raise ExqError(EXQ_ERR_INVALID_ARG, "MoeLayer")
        self.gate, self.up, self.down, self.router = gate, up, down, router
        self._desc = exq_moe_layer(gate._desc, up._desc, down._desc, None if router is None else router.data_ptr(), top_k,
                                   int(renorm), act)
        self._ref = ctypes.byref(self._desc)
        self._space = {}


def exq_moe_workspace_size(layer: MoeLayer, T: int) -> int:
    return int(_lib.exq_moe_workspace_size(layer._ref, T))


def exq_moe(layer: MoeLayer, x, ids=None, weights=None, out=None, workspace=None, stream=None):
    """(y fp16 [T, D], ids int32 [T, top_k], weights fp32 [T, top_k]) of up to 16 tokens x fp16 [T, D]. ids and weights are filled
    where the layer has a router, and read, so that both must be given, where it has none. The workspace is as exq_fp4_gemv's."""
    import torch
    where = "exq_moe"
    dev = layer.device
    _here(where, dev, x.get_device())
    if not _is_rows(x, torch.float16) or x.shape[1] != layer.D or (layer.router is None and (ids is None or weights is None)):
        raise ExqError(EXQ_ERR_INVALID_ARG, where)
    T = x.shape[0]
    shape = (T, layer.top_k)
    if ids is None:
        ids = _empty(shape, torch.int32, x.device, stream)
    elif ids.dtype is not torch.int32 or ids.shape != shape or not ids.is_contiguous() or ids.get_device() != dev:
        raise ExqError(EXQ_ERR_INVALID_ARG, where)
    if weights is None:
        weights = _empty(shape, torch.float32, x.device, stream)
    elif weights.dtype is not torch.float32 or weights.shape != shape or not weights.is_contiguous() or weights.get_device() != dev:
        raise ExqError(EXQ_ERR_INVALID_ARG, where)
    out = _result(out, T, layer.D, dev, x, stream, where)
    handle = _stream_ptr(stream, dev)
    if workspace is None:
        need = layer._space.get(T)
        if need is None:
            need = layer._space[T] = _lib.exq_moe_workspace_size(layer._ref, T)
        with _fp4_lock(dev, handle):
            _kept, ws, n = _fp4_workspace(need, dev, stream, handle, where)
            status = _lib.exq_moe(layer._ref, x.data_ptr(), T, ids.data_ptr(), weights.data_ptr(), out.data_ptr(), ws, n, handle)
    else:
        ws, n = _space(workspace, dev, where)
        status = _lib.exq_moe(layer._ref, x.data_ptr(), T, ids.data_ptr(), weights.data_ptr(), out.data_ptr(), ws, n, handle)
    _check(status, where)
    return out, ids, weights


def _i32(a, where: str) -> np.ndarray:
    if not isinstance(a, np.ndarray) or a.dtype != np.int32 or not a.flags.c_contiguous:
        raise ExqError(EXQ_ERR_INVALID_ARG, where)
    return a


def exq_pages_alloc(refs: np.ndarray, n: int) -> np.ndarray:
    """Host: the n lowest free pages of refs int32 [pages], now held once."""
    out = np.empty(max(n, 0), dtype=np.int32)
    _check(_lib.exq_pages_alloc(_np_ptr(_i32(refs, "exq_pages_alloc")), refs.size, n, _np_ptr(out)), "exq_pages_alloc")
    return out


def exq_pages_free(refs: np.ndarray, ids) -> None:
    """Host: gives up one hold on each page of ids."""
    ids = np.ascontiguousarray(ids, dtype=np.int32)
    _check(_lib.exq_pages_free(_np_ptr(_i32(refs, "exq_pages_free")), refs.size, _np_ptr(ids), ids.size), "exq_pages_free")


def exq_pages_fork(refs: np.ndarray, ids, n_tokens: int, page_size: int):
    """Host: (page ids of a second sequence sharing the first n_tokens, pairs int32 [0 or 1, 2] to copy)."""
    ids = np.ascontiguousarray(ids, dtype=np.int32)
    n = -(-n_tokens // page_size) if page_size > 0 and n_tokens > 0 else 0
    if ids.size < n:
        raise ExqError(EXQ_ERR_INVALID_ARG, "exq_pages_fork")
    out, pair, count = np.empty(n, np.int32), np.empty((1, 2), np.int32), ctypes.c_int32()
    _check(_lib.exq_pages_fork(_np_ptr(_i32(refs, "exq_pages_fork")), refs.size, page_size, _np_ptr(ids), n_tokens,
                               _np_ptr(out), _np_ptr(pair), ctypes.byref(count)), "exq_pages_fork")
    return out, pair[:count.value]


def exq_pages_compact(refs: np.ndarray, tables: np.ndarray) -> np.ndarray:
    """Host: moves the held pages to the lowest ids in refs and tables (int32, both rewritten); the pairs int32 [n, 2] to
    copy."""
    where = "exq_pages_compact"
    pairs, count = np.empty((max(refs.size // 2, 1), 2), np.int32), ctypes.c_int32()
    _check(_lib.exq_pages_compact(_np_ptr(_i32(refs, where)), refs.size, _np_ptr(_i32(tables, where)), tables.size,
                                  _np_ptr(pairs), ctypes.byref(count)), where)
    return pairs[:count.value]


def exq_solve_exl2_bits(err: np.ndarray, budget: int) -> np.ndarray:
    """Host: widths uint8 [S] for an error table float64 [S, 6] and a budget of
    code bits per column."""
    err = np.ascontiguousarray(err, dtype=np.float64)
    S = err.shape[0]
    out = np.empty(S, dtype=np.uint8)
    _check(_lib.exq_solve_exl2_bits(_np_ptr(err), S, int(budget), _np_ptr(out)), "exq_solve_exl2_bits")
    return out


def exq_measure_exl2(W, perm=None, stream=None):
    """RTN error table fp32 [K/32, 6] of an fp16 weight [K, N] (device)."""
    import torch
    K, N = W.shape
    err = _empty((K // 32, 6), torch.float32, W.device, stream)
    nws = int(_lib.exq_measure_exl2_workspace_size(K, N))
    ws = _empty(max(nws, 16), torch.uint8, W.device, stream)
    _check(_lib.exq_measure_exl2(W.data_ptr(), None if perm is None else perm.data_ptr(), K, N, err.data_ptr(),
                                 ws.data_ptr(), nws, _stream_ptr(stream)), "exq_measure_exl2")
    return err


def exq_quantize_exl2(W, bits, perm=None, stream=None) -> Weight:
    """RTN conversion of an fp16 weight [K, N] (device) at the given widths
    [K/32] into an EXL2 layer."""
    import torch
    K, N = W.shape
    off = exq_exl2_seg_word_off(bits)
    rows = int(off[-1])
    off_d = torch.from_numpy(off.view(np.int32)).to(W.device)
    qw = _empty((rows, N), torch.int32, W.device, stream)
    sc = _empty((K // 32, N), torch.float16, W.device, stream)
    _check(_lib.exq_quantize_exl2(W.data_ptr(), None if perm is None else perm.data_ptr(), K, N, off_d.data_ptr(),
                                  rows, qw.data_ptr(), sc.data_ptr(), _stream_ptr(stream)), "exq_quantize_exl2")
    return Weight(EXQ_FMT_EXL2, K, N, 32, qw, sc, None, perm, off_d)


def exq_get_last_device_error(stream=None) -> int:
    st = int(_lib.exq_get_last_device_error(_stream_ptr(stream)))
    if st == EXQ_ERR_TIMEOUT:  # calls that gave up may have left counters: the next ones of the 4-bit products get new workspaces
        for key in list(_fp4_ws):
            with _fp4_lock(*key):
                _fp4_ws.pop(key, None)
    return st


def exq_testing_starve(wait_rounds: int) -> None:
    """Failure-detection test hook (include/exq_testing.h): while wait_rounds
    > 0, launches of GEMV, GEMM, paged attention, the 4-bit products and
    the experts issue no copies and their bounded waits give up after
    wait_rounds rounds, so the call ends in EXQ_ERR_TIMEOUT; 0 = off."""
    _lib.exq_testing_starve(int(wait_rounds))
