"""ctypes binding over libwq.so: argument marshalling only.

Every call goes straight to the C ABI declared in include/wq.h; the kernels do
all of the work. PyTorch provides device memory and the current CUDA stream.
There is no fallback: if libwq.so is missing the import of a call fails.
"""

from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG_DIR, "libwq.so")

WQ_OK, WQ_EINVAL, WQ_EUNSUPPORTED, WQ_ECUDA, WQ_ETIMEOUT = range(5)
_STATUS_NAMES = {0: "WQ_OK", 1: "WQ_EINVAL", 2: "WQ_EUNSUPPORTED", 3: "WQ_ECUDA", 4: "WQ_ETIMEOUT"}

_c_i64 = ctypes.c_int64
_c_int = ctypes.c_int
_c_size = ctypes.c_size_t
_c_ptr = ctypes.c_void_p

# name -> (restype, argtypes); mirrors include/wq.h
SIGNATURES = {
    "wq_packed_words_per_row": (_c_size, [_c_i64, _c_int]),
    "wna16_repack": (_c_int, [_c_ptr, _c_ptr, _c_i64, _c_i64, _c_int, _c_int, _c_ptr, _c_ptr, _c_ptr, _c_ptr]),
    "wna16_workspace_bytes": (_c_size, [_c_i64, _c_i64, _c_i64, _c_int]),
    "wna16_gemm": (_c_int, [_c_ptr, _c_i64, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_int, _c_int, _c_ptr,
                            _c_ptr, _c_size, _c_ptr]),
    "wna16_gemm_zp": (_c_int, [_c_ptr, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_int, _c_int, _c_ptr,
                               _c_ptr, _c_size, _c_ptr]),
    "wna16_zp_workspace_bytes": (_c_size, [_c_i64, _c_i64, _c_i64, _c_int]),
    "wna16_moe_gemm": (_c_int, [_c_ptr, _c_i64, _c_ptr, _c_i64, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_int, _c_int,
                                _c_ptr, _c_ptr]),
    "wna16_gemm_noalloc": (_c_int, [_c_ptr, _c_i64, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_int, _c_int,
                                    _c_ptr, _c_ptr]),
    "act_quant_int8": (_c_int, [_c_ptr, _c_i64, _c_i64, _c_ptr, _c_ptr, _c_ptr]),
    "w4a8_workspace_bytes": (_c_size, [_c_i64, _c_i64, _c_i64]),
    "w4a8_scratch_bytes": (_c_size, [_c_i64, _c_i64]),
    "w4a8_gemm": (_c_int, [_c_ptr, _c_i64, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_int, _c_ptr, _c_ptr,
                           _c_size, _c_ptr, _c_size, _c_ptr]),
    "qembed_gather": (_c_int, [_c_ptr, _c_i64, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_int, _c_int, _c_ptr,
                               _c_ptr, _c_ptr]),
    "kv_append": (_c_int, [_c_ptr, _c_ptr, _c_i64, _c_i64, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_ptr,
                           _c_int, _c_i64, _c_i64, _c_i64, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_ptr]),
    "kv_attn_workspace_bytes": (_c_size, [_c_i64, _c_i64, _c_i64, _c_i64]),
    "kv_attn_decode": (_c_int, [_c_ptr, _c_i64, _c_ptr, _c_int, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_i64, _c_i64,
                                _c_i64, _c_i64, _c_i64, _c_ptr, _c_ptr, ctypes.c_float, _c_i64, _c_ptr, _c_ptr,
                                _c_ptr, _c_ptr, _c_size, _c_ptr]),
    "kv_pages_scratch_bytes": (_c_size, [_c_i64, _c_i64, _c_i64, _c_i64]),
    "kv_pages_copy": (_c_int, [_c_ptr, _c_i64, _c_i64, _c_i64, _c_ptr, _c_ptr, _c_i64, _c_ptr, _c_ptr]),
    "kv_pages_fork": (_c_int, [_c_ptr, _c_i64, _c_i64, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_i64,
                               _c_ptr, _c_ptr, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_size, _c_ptr]),
    "kv_pages_reserve": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_i64, _c_i64, _c_ptr, _c_ptr,
                                  _c_ptr, _c_ptr, _c_size, _c_ptr]),
    "kv_pages_free": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_i64, _c_i64, _c_ptr, _c_i64, _c_ptr,
                               _c_ptr, _c_ptr, _c_ptr]),
    "kv_pages_compact": (_c_int, [_c_ptr, _c_i64, _c_i64, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_i64,
                                  _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_size, _c_ptr]),
    "token_logprobs_workspace_bytes": (_c_size, [_c_i64, _c_i64, _c_int]),
    "token_logprobs": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_i64, _c_ptr, ctypes.c_float, _c_int, _c_ptr,
                                _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_size, _c_ptr]),
    "moe_route": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_int, ctypes.c_float, _c_ptr,
                           _c_ptr, _c_ptr]),
    "moe_route_grad": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_int, ctypes.c_float,
                                _c_ptr, _c_ptr, _c_ptr, _c_ptr]),
    "moe_sort": (_c_int, [_c_ptr, _c_i64, _c_i64, _c_i64, _c_ptr, _c_int, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_ptr,
                          _c_ptr]),
    "moe_combine": (_c_int, [_c_ptr, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_int, _c_ptr, _c_ptr]),
    "moe_combine_grad": (_c_int, [_c_ptr, _c_ptr, _c_i64, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_int, _c_ptr, _c_ptr,
                                  _c_ptr]),
    "lora_workspace_bytes": (_c_size, [_c_i64, _c_i64, _c_i64]),
    "lora_gemm": (_c_int, [_c_ptr, _c_i64, _c_i64, _c_i64, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_i64, _c_ptr, _c_ptr,
                           _c_ptr, _c_i64, _c_ptr, _c_i64, _c_ptr, _c_size, _c_ptr]),
    "wq_debug_decode_plan": (_c_int, [_c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_ptr]),
    "wq_debug_route": (_c_int, [_c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_int, _c_ptr]),
    "wq_debug_unpack": (_c_int, [_c_ptr, _c_i64, _c_i64, _c_int, _c_ptr, _c_ptr]),
    "wq_debug_w4a8_group_acc": (_c_int, [_c_ptr, _c_i64, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_ptr, _c_ptr,
                                         _c_size, _c_ptr]),
    "wq_debug_noalloc_scratch": (_c_int, [_c_ptr, _c_size, _c_int, _c_ptr]),
    "wq_debug_mma_peak": (_c_int, [_c_int, _c_i64, _c_int, _c_ptr, _c_ptr]),
    "wq_debug_decode_wait_fault": (_c_int, [_c_i64, ctypes.c_uint64]),
    "wq_check_status": (_c_int, []),
    "wq_last_error": (ctypes.c_char_p, []),
    "wq_version": (ctypes.c_char_p, []),
}

_lib = None
_lib_lock = threading.Lock()


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libwq.so (once) and attaches the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    with _lib_lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(
                    f"libwq.so not found at {path}; build it first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib  # complete before another thread can see it
        return _lib


class WQError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: {_STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def _check(status: int, where: str) -> None:
    if status != WQ_OK:
        msg = load().wq_last_error().decode()
        if status in (WQ_ECUDA, WQ_ETIMEOUT):
            # device work may have stopped part-way: a zero-at-rest workspace
            # can hold partial sums, so the cached buffers are dropped and the
            # next call gets a zero-filled one (argument errors launch nothing)
            drop_workspaces()
        raise WQError(status, where, msg)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


# The current device and stream as numbers: what torch.cuda.current_stream()
# wraps, at a fraction of its cost (a small call takes as long on the host as on
# the GPU).
def _device() -> int:
    return torch._C._cuda_getDevice()


def _stream() -> int:
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _need(t: torch.Tensor, name: str, dtype, shape=None) -> None:
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")


# ---------------------------------------------------------------- workspaces

_ws_cache: dict = {}
_ws_captured: list = []  # buffers that captured graphs use: they outlive their place in the cache
_ws_lock = threading.Lock()


def _cached(kind: str, nbytes: int, device=None) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    index = _device() if device is None else torch.device(device).index
    key = (kind, index, _stream())
    buf = _ws_cache.get(key)
    if buf is not None and buf.numel() >= nbytes:
        return buf
    with _ws_lock:
        buf = _ws_cache.get(key)
        if buf is None or buf.numel() < nbytes:
            dev = "cuda" if index is None else torch.device("cuda", index)
            buf = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=dev)
            _ws_cache[key] = buf
        return buf


def drop_workspaces() -> None:
    """Forgets every cached workspace and scratch buffer; later calls allocate
    fresh zero-filled ones. Called after a device-side failure. The memory
    returns to PyTorch's allocator, which reuses it in stream order: graphs
    captured before are not to be replayed any more."""
    with _ws_lock:
        _ws_cache.clear()
        _ws_captured.clear()


def workspace(nbytes: int, device=None) -> torch.Tensor | None:
    """A zero-filled split-K workspace for the current stream, reused across
    calls. The library leaves it zero-filled after every successful call;
    calls that share it are serialised by the stream. One that a captured call
    uses is kept for the graph when a larger one takes its place."""
    buf = _cached("zero-at-rest", nbytes, device)
    if buf is not None and torch.cuda.is_current_stream_capturing():
        with _ws_lock:
            if not any(b is buf for b in _ws_captured):
                _ws_captured.append(buf)
    return buf


def scratch(nbytes: int, device=None) -> torch.Tensor | None:
    """A scratch buffer (contents undefined between calls) for the current stream.
    A call that is captured into a CUDA graph gets one of its own from the
    graph's memory: a cached one could be replaced, or be in use by another
    graph, when the graph runs."""
    if nbytes and torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device="cuda" if device is None else device)
    return _cached("scratch", nbytes, device)


# ---------------------------------------------------------------- host queries

def packed_words_per_row(K: int, bits: int) -> int:
    return int(load().wq_packed_words_per_row(K, bits))


def wna16_workspace_bytes(M: int, N: int, K: int, bits: int) -> int:
    return int(load().wna16_workspace_bytes(M, N, K, bits))


def wna16_zp_workspace_bytes(M: int, N: int, K: int, bits: int) -> int:
    return int(load().wna16_zp_workspace_bytes(M, N, K, bits))


def w4a8_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load().w4a8_workspace_bytes(M, N, K))


def w4a8_scratch_bytes(M: int, K: int) -> int:
    return int(load().w4a8_scratch_bytes(M, K))


def version() -> str:
    return load().wq_version().decode()


def check_status() -> None:
    _check(load().wq_check_status(), "wq_check_status")


# ---------------------------------------------------------------- entry points

def wna16_repack(codes: torch.Tensor, scales: torch.Tensor, bits: int, group: int = 128,
                 packed: torch.Tensor | None = None, scales_out: torch.Tensor | None = None,
                 bad_count: torch.Tensor | None = None):
    """codes uint8 [N, K], scales bf16 [N, K/128] -> (packed uint32-as-int32 [N, W], scales_out)."""
    N, K = codes.shape
    _need(codes, "codes", torch.uint8)
    _need(scales, "scales", torch.bfloat16, (N, K // group))
    W = packed_words_per_row(K, bits)
    if packed is None:
        packed = torch.empty((N, W), dtype=torch.int32, device=codes.device)
    _need(packed, "packed", torch.int32, (N, W))
    if scales_out is None:
        scales_out = torch.empty_like(scales)
    _need(scales_out, "scales_out", torch.bfloat16, (N, K // group))
    if bad_count is not None:
        _need(bad_count, "bad_count", torch.int32)
    _check(load().wna16_repack(_ptr(codes), _ptr(scales), N, K, bits, group, _ptr(packed),
                               _ptr(scales_out), _ptr(bad_count), _stream()), "wna16_repack")
    return packed, scales_out


def wna16_gemm(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, N: int, K: int, bits: int,
               group: int = 128, y: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """y[M, N] = x[M, K] . dequant(W)^T, bf16 out."""
    M = x.shape[0]
    _need(x, "x", torch.bfloat16, (M, K))
    _need(packed, "packed", torch.int32, (N, packed_words_per_row(K, bits)))
    _need(scales, "scales", torch.bfloat16, (N, K // group))
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _need(y, "y", torch.bfloat16, (M, N))
    need = wna16_workspace_bytes(M, N, K, bits)
    if ws is None:
        ws = workspace(need)
    _check(load().wna16_gemm(_ptr(x), M, _ptr(packed), _ptr(scales), N, K, bits, group, _ptr(y),
                             _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _stream()),
           "wna16_gemm")
    return y


def wna16_gemm_zp(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, N: int,
                  K: int, bits: int, group: int = 128, y: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None):
    """y[M, N] = x[M, K] . dequant(W)^T with a zero point per (row, group):
    w = s * (q - zp); zeros uint8 [N, K/128]."""
    M = x.shape[0]
    _need(x, "x", torch.bfloat16, (M, K))
    _need(packed, "packed", torch.int32, (N, packed_words_per_row(K, bits)))
    _need(scales, "scales", torch.bfloat16, (N, K // group))
    _need(zeros, "zeros", torch.uint8, (N, K // group))
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _need(y, "y", torch.bfloat16, (M, N))
    need = wna16_zp_workspace_bytes(M, N, K, bits)
    if ws is None:
        ws = workspace(need)
    _check(load().wna16_gemm_zp(_ptr(x), M, _ptr(packed), _ptr(scales), _ptr(zeros), N, K, bits, group, _ptr(y),
                                _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _stream()),
           "wna16_gemm_zp")
    return y


def wna16_moe_gemm(x: torch.Tensor, expert_offsets: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                   E: int, N: int, K: int, bits: int, group: int = 128, y: torch.Tensor | None = None):
    """Mixture of experts: x [M, K] sorted by expert, expert_offsets int32
    [E + 1] on the device, packed [E * N, words] and scales [E * N, K/128]
    stacked per expert; y [M, N]."""
    M = x.shape[0]
    _need(x, "x", torch.bfloat16, (M, K))
    _need(expert_offsets, "expert_offsets", torch.int32, (E + 1,))
    _need(packed, "packed", torch.int32, (E * N, packed_words_per_row(K, bits)))
    _need(scales, "scales", torch.bfloat16, (E * N, K // group))
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _need(y, "y", torch.bfloat16, (M, N))
    _check(load().wna16_moe_gemm(_ptr(x), M, _ptr(expert_offsets), E, _ptr(packed), _ptr(scales), N, K, bits, group,
                                 _ptr(y), _stream()), "wna16_moe_gemm")
    return y


def wna16_gemm_noalloc(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, N: int, K: int,
                       bits: int, group: int = 128, y: torch.Tensor | None = None):
    """wna16_gemm without a workspace: the library's fixed scratch array is
    used instead (for callers that cannot allocate device memory)."""
    M = x.shape[0]
    _need(x, "x", torch.bfloat16, (M, K))
    _need(packed, "packed", torch.int32, (N, packed_words_per_row(K, bits)))
    _need(scales, "scales", torch.bfloat16, (N, K // group))
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _need(y, "y", torch.bfloat16, (M, N))
    _check(load().wna16_gemm_noalloc(_ptr(x), M, _ptr(packed), _ptr(scales), N, K, bits, group, _ptr(y),
                                     _stream()), "wna16_gemm_noalloc")
    return y


def act_quant_int8(x: torch.Tensor, xq: torch.Tensor | None = None, sx: torch.Tensor | None = None):
    M, K = x.shape
    _need(x, "x", torch.bfloat16)
    if xq is None:
        xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if sx is None:
        sx = torch.empty((M,), dtype=torch.float32, device=x.device)
    _need(xq, "xq", torch.int8, (M, K))
    _need(sx, "sx", torch.float32, (M,))
    _check(load().act_quant_int8(_ptr(x), M, K, _ptr(xq), _ptr(sx), _stream()), "act_quant_int8")
    return xq, sx


def w4a8_gemm(x: torch.Tensor, packed4: torch.Tensor, scales: torch.Tensor, N: int, K: int,
              group: int = 128, y: torch.Tensor | None = None, ws: torch.Tensor | None = None,
              scr: torch.Tensor | None = None):
    M = x.shape[0]
    _need(x, "x", torch.bfloat16, (M, K))
    _need(packed4, "packed4", torch.int32, (N, packed_words_per_row(K, 4)))
    _need(scales, "scales", torch.bfloat16, (N, K // group))
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _need(y, "y", torch.bfloat16, (M, N))
    need = w4a8_workspace_bytes(M, N, K)
    if ws is None:
        ws = workspace(need)
    if scr is None:
        scr = scratch(w4a8_scratch_bytes(M, K))
    _check(load().w4a8_gemm(_ptr(x), M, _ptr(packed4), _ptr(scales), N, K, group, _ptr(y), _ptr(ws),
                            0 if ws is None else ws.numel() * ws.element_size(), _ptr(scr),
                            scr.numel() * scr.element_size(), _stream()), "w4a8_gemm")
    return y


def qembed_gather(ids: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, V: int, D: int,
                  bits: int, group: int = 128, out: torch.Tensor | None = None,
                  bad_count: torch.Tensor | None = None):
    T = ids.shape[0]
    _need(ids, "ids", torch.int32, (T,))
    _need(packed, "packed", torch.int32, (V, packed_words_per_row(D, bits)))
    _need(scales, "scales", torch.bfloat16, (V, D // group))
    if out is None:
        out = torch.empty((T, D), dtype=torch.bfloat16, device=ids.device)
    _need(out, "out", torch.bfloat16, (T, D))
    if bad_count is not None:
        _need(bad_count, "bad_count", torch.int32)
    _check(load().qembed_gather(_ptr(ids), T, _ptr(packed), _ptr(scales), V, D, bits, group, _ptr(out),
                                _ptr(bad_count), _stream()), "qembed_gather")
    return out


# ---------------------------------------------------------------- serving operators

_KV_TYPES = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}
_LOGIT_TYPES = {torch.bfloat16: 0, torch.float32: 1}


def _need_rows(t: torch.Tensor, name: str, shape) -> int:
    """A bf16 tensor whose rows are contiguous and whose first dimension may
    have any stride; returns that stride in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16 (got {t.dtype})")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    row = shape[1] * shape[2]
    if shape[0] == 0:
        return row
    if t.stride(2) != 1 or (shape[1] > 1 and t.stride(1) != shape[2]):
        raise ValueError(f"each row of {name} must be contiguous")
    return row if shape[0] == 1 else t.stride(0)


def _need_cache(kv: torch.Tensor, k_scale, v_scale):
    if not isinstance(kv, torch.Tensor) or kv.dim() != 5 or kv.shape[1] != 2:
        raise ValueError("kv must be a tensor [P, 2, Hkv, S, D]")
    if kv.dtype not in _KV_TYPES:
        raise TypeError(f"kv must be bfloat16 or float8_e4m3fn (got {kv.dtype})")
    _need(kv, "kv", kv.dtype)
    if kv.dtype == torch.bfloat16:
        if k_scale is not None or v_scale is not None:
            raise ValueError("k_scale and v_scale are for e4m3 caches")
    else:
        _need(k_scale, "k_scale", torch.float32, (kv.shape[2],))
        _need(v_scale, "v_scale", torch.float32, (kv.shape[2],))
    return _KV_TYPES[kv.dtype]


def _need_pool(kv: torch.Tensor):
    """kv [L, P, 2, Hkv, S, D] or one layer's [P, 2, Hkv, S, D]: (L, P, S, page bytes)."""
    if not isinstance(kv, torch.Tensor) or kv.dim() not in (5, 6) or kv.shape[-4] != 2:
        raise ValueError("kv must be a tensor [L, P, 2, Hkv, S, D] or [P, 2, Hkv, S, D]")
    if kv.dtype not in _KV_TYPES:
        raise TypeError(f"kv must be bfloat16 or float8_e4m3fn (got {kv.dtype})")
    _need(kv, "kv", kv.dtype)
    L, (P, two, H, S, D) = (kv.shape[0] if kv.dim() == 6 else 1), kv.shape[-5:]
    return L, P, S, two * H * S * D * kv.element_size()


@functools.lru_cache(maxsize=4096)
def kv_attn_workspace_bytes(B: int, Hq: int, Hkv: int, D: int) -> int:
    return int(load().kv_attn_workspace_bytes(B, Hq, Hkv, D))


@functools.lru_cache(maxsize=4096)
def kv_pages_scratch_bytes(n: int, B: int, W: int, P: int) -> int:
    return int(load().kv_pages_scratch_bytes(n, B, W, P))


@functools.lru_cache(maxsize=4096)
def token_logprobs_workspace_bytes(T: int, V: int, top_k: int) -> int:
    return int(load().token_logprobs_workspace_bytes(T, V, top_k))


def kv_append(k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor, block_table: torch.Tensor, kv: torch.Tensor,
              seq: torch.Tensor | None = None, k_scale: torch.Tensor | None = None,
              v_scale: torch.Tensor | None = None, bad_count: torch.Tensor | None = None) -> torch.Tensor:
    """Writes k, v [T, Hkv, D] bf16 (rows may be strided) into the pages of kv
    [P, 2, Hkv, S, D]: token t as token pos[t] of sequence seq[t] (of sequence
    t without seq). Returns kv."""
    kind = _need_cache(kv, k_scale, v_scale)
    P, _, H, S, D = kv.shape
    T, (B, W) = k.shape[0], block_table.shape
    ks, vs = _need_rows(k, "k", (T, H, D)), _need_rows(v, "v", (T, H, D))
    _need(pos, "pos", torch.int32, (T,))
    _need(block_table, "block_table", torch.int32, (B, W))
    if seq is not None:
        _need(seq, "seq", torch.int32, (T,))
    if bad_count is not None:
        _need(bad_count, "bad_count", torch.int32)
    _check(load().kv_append(k.data_ptr(), v.data_ptr(), ks, vs, T, _ptr(seq), pos.data_ptr(),
                            block_table.data_ptr(), B, W, kv.data_ptr(), kind, P, H, S, D, _ptr(k_scale),
                            _ptr(v_scale), _ptr(bad_count), _stream()), "kv_append")
    return kv


def kv_attn_decode(q: torch.Tensor, kv: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor,
                   sm_scale: float | None = None, window: int = 0, k_scale: torch.Tensor | None = None,
                   v_scale: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, return_lse: bool = False,
                   bad_count: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """Attention of one new token per sequence: q [B, Hq, D] bf16 over the
    lens[b] tokens of kv [P, 2, Hkv, S, D] that block_table [B, W] names.
    sm_scale: 1/sqrt(D) if None; window: the last so many tokens (0: all).
    Returns out [B, Hq, D] bf16, and lse [B, Hq] float32 with return_lse."""
    kind = _need_cache(kv, k_scale, v_scale)
    P, _, H, S, D = kv.shape
    B, Hq = q.shape[0], q.shape[1]
    W = block_table.shape[1]
    qs = _need_rows(q, "q", (B, Hq, D))
    _need(block_table, "block_table", torch.int32, (B, W))
    _need(lens, "lens", torch.int32, (B,))
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=q.device)
    else:
        _need(out, "out", torch.bfloat16, (B, Hq, D))
    if lse is not None:
        _need(lse, "lse", torch.float32, (B, Hq))
    elif return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if bad_count is not None:
        _need(bad_count, "bad_count", torch.int32)
    lib = load()
    if ws is None:
        ws = scratch(kv_attn_workspace_bytes(B, Hq, H, D))
    _check(lib.kv_attn_decode(q.data_ptr(), qs, kv.data_ptr(), kind, block_table.data_ptr(), lens.data_ptr(), B, W,
                              P, Hq, H, S, D, _ptr(k_scale), _ptr(v_scale), D ** -0.5 if sm_scale is None else
                              sm_scale, window, out.data_ptr(), _ptr(lse), _ptr(bad_count), _ptr(ws), 0 if ws is
                              None else ws.numel() * ws.element_size(), _stream()), "kv_attn_decode")
    return (out, lse) if return_lse else out


def kv_pages_copy(kv: torch.Tensor, src: torch.Tensor, dst: torch.Tensor,
                  bad_count: torch.Tensor | None = None) -> torch.Tensor:
    """Copies page src[i] to page dst[i] in every layer of kv; returns kv."""
    L, P, _, size = _need_pool(kv)
    n = src.shape[0]
    _need(src, "src", torch.int32, (n,))
    _need(dst, "dst", torch.int32, (n,))
    if bad_count is not None:
        _need(bad_count, "bad_count", torch.int32)
    _check(load().kv_pages_copy(kv.data_ptr(), L, P, size, src.data_ptr(), dst.data_ptr(), n, _ptr(bad_count),
                                _stream()), "kv_pages_copy")
    return kv


def _need_tables(block_table, lens, ref):
    B, W = block_table.shape
    P = ref.shape[0]
    _need(block_table, "block_table", torch.int32, (B, W))
    _need(lens, "lens", torch.int32, (B,))
    _need(ref, "ref", torch.int32, (P,))
    return B, W, P


def _or_in_place(out, given, name):
    if out is None:
        return given
    _need(out, name, torch.int32, given.shape)
    return out


def _out_32(out, shape, name, device):
    if out is None:
        return torch.empty(shape, dtype=torch.int32, device=device)
    _need(out, name, torch.int32, shape)
    return out


def kv_pages_fork(kv: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor, ref: torch.Tensor,
                  parent: torch.Tensor, child: torch.Tensor, table_out: torch.Tensor | None = None,
                  lens_out: torch.Tensor | None = None, ref_out: torch.Tensor | None = None,
                  granted: torch.Tensor | None = None):
    """Starts sequence child[i] as a copy of parent[i]: full pages are shared,
    a partial last page is copied to a free one. Updates block_table, lens and
    ref in place unless given other outputs; returns (block_table, lens, ref,
    granted)."""
    L, P, S, size = _need_pool(kv)
    B, W, _ = _need_tables(block_table, lens, ref)
    _need(ref, "ref", torch.int32, (P,))
    n = parent.shape[0]
    _need(parent, "parent", torch.int32, (n,))
    _need(child, "child", torch.int32, (n,))
    table_out = _or_in_place(table_out, block_table, "table_out")
    lens_out, ref_out = _or_in_place(lens_out, lens, "lens_out"), _or_in_place(ref_out, ref, "ref_out")
    granted = _out_32(granted, (n,), "granted", kv.device)
    lib = load()
    scr = scratch(kv_pages_scratch_bytes(n, B, W, P))
    _check(lib.kv_pages_fork(kv.data_ptr(), L, P, size, block_table.data_ptr(), lens.data_ptr(), ref.data_ptr(), B,
                             W, S, parent.data_ptr(), child.data_ptr(), n, table_out.data_ptr(),
                             lens_out.data_ptr(), ref_out.data_ptr(), granted.data_ptr(), _ptr(scr), scr.numel(),
                             _stream()), "kv_pages_fork")
    return table_out, lens_out, ref_out, granted


def kv_pages_reserve(block_table: torch.Tensor, lens: torch.Tensor, new_lens: torch.Tensor, ref: torch.Tensor,
                     page_size: int, table_out: torch.Tensor | None = None, ref_out: torch.Tensor | None = None,
                     granted: torch.Tensor | None = None):
    """Gives every sequence the free pages that new_lens[b] tokens need beyond
    those of lens[b]. Updates block_table and ref in place unless given other
    outputs; returns (block_table, ref, granted)."""
    B, W, P = _need_tables(block_table, lens, ref)
    _need(new_lens, "new_lens", torch.int32, (B,))
    table_out, ref_out = _or_in_place(table_out, block_table, "table_out"), _or_in_place(ref_out, ref, "ref_out")
    granted = _out_32(granted, (B,), "granted", ref.device)
    lib = load()
    scr = scratch(kv_pages_scratch_bytes(B, B, W, P))
    _check(lib.kv_pages_reserve(block_table.data_ptr(), lens.data_ptr(), new_lens.data_ptr(), ref.data_ptr(), B, W,
                                page_size, P, table_out.data_ptr(), ref_out.data_ptr(), granted.data_ptr(),
                                _ptr(scr), 0 if scr is None else scr.numel(), _stream()), "kv_pages_reserve")
    return table_out, ref_out, granted


def kv_pages_free(block_table: torch.Tensor, lens: torch.Tensor, ref: torch.Tensor, seqs: torch.Tensor,
                  page_size: int, lens_out: torch.Tensor | None = None, ref_out: torch.Tensor | None = None,
                  bad_count: torch.Tensor | None = None):
    """Gives back the pages of the sequences seqs. Updates lens and ref in
    place unless given other outputs; returns (lens, ref)."""
    B, W, P = _need_tables(block_table, lens, ref)
    n = seqs.shape[0]
    _need(seqs, "seqs", torch.int32, (n,))
    lens_out, ref_out = _or_in_place(lens_out, lens, "lens_out"), _or_in_place(ref_out, ref, "ref_out")
    if bad_count is not None:
        _need(bad_count, "bad_count", torch.int32)
    _check(load().kv_pages_free(block_table.data_ptr(), lens.data_ptr(), ref.data_ptr(), B, W, page_size, P,
                                seqs.data_ptr(), n, lens_out.data_ptr(), ref_out.data_ptr(), _ptr(bad_count),
                                _stream()), "kv_pages_free")
    return lens_out, ref_out


def kv_pages_compact(kv: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor, ref: torch.Tensor,
                     table_out: torch.Tensor | None = None, ref_out: torch.Tensor | None = None,
                     remap: torch.Tensor | None = None, n_live: torch.Tensor | None = None):
    """Moves the pages in use to the front of the pool. Updates block_table and
    ref in place unless given other outputs; returns (block_table, ref, remap,
    n_live)."""
    L, P, S, size = _need_pool(kv)
    B, W, _ = _need_tables(block_table, lens, ref)
    _need(ref, "ref", torch.int32, (P,))
    table_out, ref_out = _or_in_place(table_out, block_table, "table_out"), _or_in_place(ref_out, ref, "ref_out")
    remap, n_live = _out_32(remap, (P,), "remap", kv.device), _out_32(n_live, (1,), "n_live", kv.device)
    lib = load()
    scr = scratch(kv_pages_scratch_bytes(0, B, W, P))
    _check(lib.kv_pages_compact(kv.data_ptr(), L, P, size, block_table.data_ptr(), lens.data_ptr(), ref.data_ptr(),
                                B, W, S, table_out.data_ptr(), ref_out.data_ptr(), remap.data_ptr(),
                                n_live.data_ptr(), _ptr(scr), scr.numel(), _stream()), "kv_pages_compact")
    return table_out, ref_out, remap, n_live


def token_logprobs(logits: torch.Tensor, ids: torch.Tensor | None = None, top_k: int = 0, temperature: float = 1.0,
                   bad_count: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """Per row of logits [T, V] (bf16 or float32, rows may be strided by any
    number, the first logit 16-byte aligned): the log probability and rank of ids[t], the entropy, and the best top_k tokens.
    Returns (logprob [T], rank [T], entropy [T], top_logprobs [T, top_k],
    top_ids [T, top_k]); logprob and rank are None without ids."""
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    if logits.dtype not in _LOGIT_TYPES:
        raise TypeError(f"logits must be bfloat16 or float32 (got {logits.dtype})")
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be [T, V] with contiguous rows")
    (T, V), dev = logits.shape, logits.device
    lp = rank = None
    if ids is not None:
        _need(ids, "ids", torch.int32, (T,))
        lp = torch.empty(T, dtype=torch.float32, device=dev)
        rank = torch.empty(T, dtype=torch.int32, device=dev)
    if bad_count is not None:
        _need(bad_count, "bad_count", torch.int32)
    k = max(int(top_k), 0)
    entropy = torch.empty(T, dtype=torch.float32, device=dev)
    top = torch.empty((T, k), dtype=torch.float32, device=dev)
    top_ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    lib = load()
    if ws is None:
        ws = scratch(token_logprobs_workspace_bytes(T, V, k))
    _check(lib.token_logprobs(logits.data_ptr(), _LOGIT_TYPES[logits.dtype], V if T <= 1 else logits.stride(0), T,
                              V, _ptr(ids), temperature, top_k, _ptr(lp), _ptr(rank), entropy.data_ptr(),
                              top.data_ptr(), top_ids.data_ptr(), _ptr(bad_count), _ptr(ws), 0 if ws is None else
                              ws.numel() * ws.element_size(), _stream()), "token_logprobs")
    return lp, rank, entropy, top, top_ids


# ---------------------------------------------------------------- operators that pick weights by token

_SCORES = {"softmax": 0, "sigmoid": 1}
_LOGIT_DTYPES = tuple(_LOGIT_TYPES)


def _need_here(t: torch.Tensor, name: str) -> None:
    """A tensor on the current device: the call's kernels run there, on its current stream."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    at = t.get_device()
    if at < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    dev = _device()
    if at != dev:
        raise ValueError(f"{name} is on cuda:{at}, the current device is cuda:{dev}")


def _need_at(t: torch.Tensor, name: str, dtype, shape=None) -> None:
    _need_here(t, name)
    _need(t, name, dtype, shape)


def _need_matrix(t: torch.Tensor, name: str, shape, dtypes=(torch.bfloat16,)) -> int:
    """A matrix whose rows are contiguous and may lie any stride apart; returns that stride in elements."""
    _need_here(t, name)
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)} (got {t.dtype})")
    got, strides = t.shape, t.stride()
    if len(got) != 2 or (shape is not None and got != shape):
        raise ValueError(f"{name} must have {'two dimensions' if shape is None else f'shape {tuple(shape)}'} (got {tuple(got)})")
    rows, cols = got
    if cols > 1 and strides[1] != 1 and rows > 0:
        raise ValueError(f"each row of {name} must be contiguous")
    return cols if rows <= 1 else strides[0]


def _score(score: str) -> int:
    if score not in _SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid' (got {score!r})")
    return _SCORES[score]


def _or_new(out, name, dtype, shape, device) -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need_at(out, name, dtype, shape)
    return out


# A small call takes longer on the host than on the GPU, and most of that were the
# checks: what passes these few comparisons passes the full checks, which are made
# (and say what is wrong) only where something does not.
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _plain(t, dtype, shape, dev) -> bool:
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev
            and t.is_contiguous())


def _tensors(*pairs) -> int:
    """Tensors (with their names) on the GPU, the first on the current device, whose number is returned."""
    for t, name in pairs:
        if not isinstance(t, torch.Tensor) or t.get_device() < 0:
            _need_here(t, name)
    _need_here(*pairs[0])
    return pairs[0][0].get_device()


def moe_route(logits: torch.Tensor, top_k: int, score: str = "softmax", renormalize: bool = False,
              scale: float = 1.0, ids: torch.Tensor | None = None, weights: torch.Tensor | None = None):
    """The top_k experts of each token by its logits [T, E] (bf16 or float32, rows may be strided) and their weights:
    scale times the softmax or sigmoid score, divided by the chosen ones' sum with renormalize. Returns (ids [T, top_k]
    int32, weights [T, top_k] float32); an expert whose logit is -inf is never chosen (id -1, weight 0)."""
    ld = _need_matrix(logits, "logits", None, _LOGIT_DTYPES)
    (T, E), dev = logits.shape, logits.device
    k = max(int(top_k), 0)
    ids = _or_new(ids, "ids", torch.int32, (T, k), dev)
    weights = _or_new(weights, "weights", torch.float32, (T, k), dev)
    _check(load().moe_route(logits.data_ptr(), _LOGIT_TYPES[logits.dtype], ld, T, E, top_k, _score(score),
                            1 if renormalize else 0, scale, ids.data_ptr(), weights.data_ptr(), _stream()), "moe_route")
    return ids, weights


def moe_route_grad(logits: torch.Tensor, ids: torch.Tensor, dweights: torch.Tensor, score: str = "softmax",
                   renormalize: bool = False, scale: float = 1.0, dlogits: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of moe_route's weights: dlogits [T, E] of the logits' type, from the ids that it returned and
    dweights [T, top_k] float32."""
    ld = _need_matrix(logits, "logits", None, _LOGIT_DTYPES)
    T, E = logits.shape
    _need_at(ids, "ids", torch.int32)
    if ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError(f"ids must have shape ({T}, top_k) (got {tuple(ids.shape)})")
    k = ids.shape[1]
    if not _plain(dweights, _F32, ids.shape, _device()):
        _need_at(dweights, "dweights", torch.float32, (T, k))
    dlogits = _or_new(dlogits, "dlogits", logits.dtype, (T, E), logits.device)
    _check(load().moe_route_grad(logits.data_ptr(), _LOGIT_TYPES[logits.dtype], ld, T, E, k, _score(score),
                                 1 if renormalize else 0, scale, ids.data_ptr(), dweights.data_ptr(),
                                 dlogits.data_ptr(), _stream()), "moe_route_grad")
    return dlogits


def moe_sort(x: torch.Tensor | None, ids: torch.Tensor, E: int, out: torch.Tensor | None = None,
             offsets: torch.Tensor | None = None, slots: torch.Tensor | None = None,
             bad_count: torch.Tensor | None = None):
    """x [T, D] bf16 (rows may be strided) in the order of the experts ids [T, k] int32, as wna16_moe_gemm reads it.
    Returns (out [T * k, D], offsets [E + 1] int32, slots [T, k] int32, the row of each choice, -1 without an expert);
    rows of out that no choice takes stay as they are. x None: out is None. The gradient of x is
    moe_combine(dout, slots)."""
    _need_at(ids, "ids", torch.int32)
    shape = ids.shape
    if len(shape) != 2:
        raise ValueError(f"ids must be [T, k] (got {tuple(shape)})")
    (T, k), dev = shape, ids.device
    D = xs = 0
    if x is not None:
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            raise ValueError("x must be a tensor [T, D]")
        D = x.shape[1]
        xs = _need_matrix(x, "x", (T, D))
        if out is None or not _plain(out, _BF16, (T * k, D), _device()):
            out = _or_new(out, "out", torch.bfloat16, (T * k, D), dev)
    elif out is not None:
        raise ValueError("out is for a call with x")
    offsets = _or_new(offsets, "offsets", torch.int32, (E + 1,), dev)
    slots = _or_new(slots, "slots", torch.int32, shape, dev)
    if bad_count is not None:
        _need_at(bad_count, "bad_count", torch.int32)
    _check(load().moe_sort(_ptr(x), xs, T, D, ids.data_ptr(), k, E, _ptr(out), offsets.data_ptr(), slots.data_ptr(),
                           _ptr(bad_count), _stream()), "moe_sort")
    return out, offsets, slots


def _rows_and_slots(y, slots):
    dev = _tensors((y, "y"), (slots, "slots"))
    ys, ss = y.shape, slots.shape
    if not _plain(y, _BF16, ys, dev):
        _need_at(y, "y", torch.bfloat16)
    if not _plain(slots, _I32, ss, dev):
        _need_at(slots, "slots", torch.int32)
    if len(ys) != 2 or len(ss) != 2:
        raise ValueError(f"y must be [R, D] and slots [T, k] (got {tuple(ys)} and {tuple(ss)})")
    return ys, ss, dev


def moe_combine(y: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None,
                residual: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """out[t] = (residual[t] +) sum_j weights[t, j] * y[slots[t, j]], [T, D] bf16: the choices' rows y [R, D] bf16
    back to their tokens (weights [T, k] float32; 1 without them). out may be residual itself."""
    (R, D), (T, k), dev = _rows_and_slots(y, slots)
    if weights is not None and not _plain(weights, _F32, (T, k), dev):
        _need_at(weights, "weights", torch.float32, (T, k))
    if residual is not None and not _plain(residual, _BF16, (T, D), dev):
        _need_at(residual, "residual", torch.bfloat16, (T, D))
    out = _or_new(out, "out", torch.bfloat16, (T, D), y.device)
    _check(load().moe_combine(y.data_ptr(), R, slots.data_ptr(), _ptr(weights), _ptr(residual), T, D, k,
                              out.data_ptr(), _stream()), "moe_combine")
    return out


def moe_combine_grad(dout: torch.Tensor, y: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor,
                     dy: torch.Tensor | None = None, dweights: torch.Tensor | None = None):
    """The gradients of moe_combine from dout [T, D] bf16: dy [R, D] bf16 (rows that no choice names stay as they
    are) and dweights [T, k] float32. The residual's is dout itself."""
    (R, D), (T, k), dev = _rows_and_slots(y, slots)
    if not _plain(dout, _BF16, (T, D), dev):
        _need_at(dout, "dout", torch.bfloat16, (T, D))
    if not _plain(weights, _F32, (T, k), dev):
        _need_at(weights, "weights", torch.float32, (T, k))
    if dy is None or not _plain(dy, _BF16, (R, D), dev):
        dy = _or_new(dy, "dy", torch.bfloat16, (R, D), y.device)
    dweights = _or_new(dweights, "dweights", torch.float32, (T, k), y.device)
    _check(load().moe_combine_grad(dout.data_ptr(), y.data_ptr(), R, slots.data_ptr(), weights.data_ptr(), T, D, k,
                                   dy.data_ptr(), dweights.data_ptr(), _stream()), "moe_combine_grad")
    return dy, dweights


@functools.lru_cache(maxsize=4096)
def lora_workspace_bytes(M: int, n: int, r: int) -> int:
    return int(load().lora_workspace_bytes(M, n, r))


def _check_lora(x, A, B, adapter, base):
    dev = _tensors((A, "A"), (B, "B"), (adapter, "adapter"))
    As, Bs = A.shape, B.shape
    if len(As) != 3 or len(Bs) != 3:
        raise ValueError(f"A must be [n, r, K] and B [n, N, r] (got {tuple(As)} and {tuple(Bs)})")
    n, r, K = As
    N, M = Bs[1], adapter.shape[0] if adapter.dim() else 0
    if not _plain(A, _BF16, As, dev):
        _need_at(A, "A", torch.bfloat16)
    if not _plain(B, _BF16, (n, N, r), dev):
        _need_at(B, "B", torch.bfloat16, (n, N, r))
    if not _plain(adapter, _I32, (M,), dev):
        _need_at(adapter, "adapter", torch.int32, (M,))
    xs, bs = _need_matrix(x, "x", (M, K)), _need_matrix(base, "base", (M, N))
    return n, r, K, N, M, xs, bs


def lora_gemm(x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, adapter: torch.Tensor, base: torch.Tensor,
              scale: torch.Tensor | None = None, y: torch.Tensor | None = None,
              ws: torch.Tensor | None = None) -> torch.Tensor:
    """y[m] = base[m] + scale[a] * (x[m] . A[a]^T) . B[a]^T with a = adapter[m] (int32; -1: none, y[m] = base[m]).
    x [M, K], base and y [M, N] bf16 (rows may be strided; y may be base), A [n, r, K], B [n, N, r] bf16, scale [n]
    float32. base is the shared projection's output, such as wna16_gemm(x, ..)."""
    try:  # (as _plain and _need_matrix, in one go: this call has the most tensors)
        (n, r, K), (_, N, _), (M,), dev = A.shape, B.shape, adapter.shape, _device()
        (xs, x1), (bs, b1) = x.stride(), base.stride()
        good = (A.dtype is _BF16 and B.dtype is _BF16 and x.dtype is _BF16 and base.dtype is _BF16 and adapter.dtype is _I32
                and B.shape == (n, N, r) and x.shape == (M, K) and base.shape == (M, N) and x1 == 1 and b1 == 1 and M > 0
                and A.get_device() == dev and B.get_device() == dev and x.get_device() == dev
                and base.get_device() == dev and adapter.get_device() == dev and A.is_contiguous()
                and B.is_contiguous() and adapter.is_contiguous())
        if M == 1:
            xs, bs = K, N
    except (AttributeError, TypeError, ValueError, RuntimeError):
        good = False
    if not good:
        n, r, K, N, M, xs, bs = _check_lora(x, A, B, adapter, base)
        dev = _device()
    if scale is not None and not _plain(scale, _F32, (n,), dev):
        _need_at(scale, "scale", torch.float32, (n,))
    if y is None:
        y, ys = torch.empty((M, N), dtype=torch.bfloat16, device=base.device), N
    else:
        ys = _need_matrix(y, "y", (M, N))
        if M <= 1 and y.data_ptr() == base.data_ptr():
            ys = bs
    lib = load()
    if ws is None:
        ws = scratch(lora_workspace_bytes(M, n, r))
    elif not (isinstance(ws, torch.Tensor) and ws.get_device() == dev and ws.is_contiguous()):
        _need_here(ws, "ws")
        raise ValueError("ws must be contiguous")
    _check(lib.lora_gemm(x.data_ptr(), xs, M, K, A.data_ptr(), B.data_ptr(), n, r, N, adapter.data_ptr(), _ptr(scale),
                         base.data_ptr(), bs, y.data_ptr(), ys, _ptr(ws), 0 if ws is None else
                         ws.numel() * ws.element_size(), _stream()), "lora_gemm")
    return y


_PLAN_KEYS = ("ok", "C", "H", "nchunk", "T", "ksplit", "NS", "G", "Gh", "sbox", "sx0", "NT", "smem",
              "max_slots")


def debug_decode_plan(M: int, N: int, K: int, bits: int, sm_count: int) -> dict:
    """The CTA-pair decode kernel's launch plan for a shape (host only)."""
    out = (ctypes.c_int64 * len(_PLAN_KEYS))()
    _check(load().wq_debug_decode_plan(M, N, K, bits, sm_count, ctypes.addressof(out)), "wq_debug_decode_plan")
    return dict(zip(_PLAN_KEYS, (int(v) for v in out)))


ROUTES = {0: "none", 1: "decode_pair", 2: "decode_splitk", 3: "chunked", 4: "tensor_core"}


def debug_route(M: int, N: int, K: int, bits: int, sm_count: int, w4a8: bool = False, zp: bool = False) -> str:
    """Which kernel wna16_gemm (or w4a8_gemm, or with zp wna16_gemm_zp)
    launches for a shape on a device with sm_count SMs (host only): one of the
    ROUTES names."""
    out = ctypes.c_int(0)
    kind = 1 if w4a8 else (2 if zp else 0)
    _check(load().wq_debug_route(M, N, K, bits, kind, sm_count, ctypes.byref(out)), "wq_debug_route")
    return ROUTES[out.value]


def debug_unpack(packed: torch.Tensor, N: int, K: int, bits: int) -> torch.Tensor:
    _need(packed, "packed", torch.int32, (N, packed_words_per_row(K, bits)))
    codes = torch.empty((N, K), dtype=torch.uint8, device=packed.device)
    _check(load().wq_debug_unpack(_ptr(packed), N, K, bits, _ptr(codes), _stream()), "wq_debug_unpack")
    return codes


def debug_mma_peak(kind: int, iters: int, blocks: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """Launches the mma.sync throughput probe (kind 0: int8 m16n8k32, kind 1:
    bf16 m16n8k16) on the current stream; returns the per-thread checksums
    [blocks * 256] int32 (each 8 * 4 * K * iters)."""
    if out is None:
        out = torch.empty(blocks * 256, dtype=torch.int32, device="cuda")
    _need(out, "out", torch.int32, (blocks * 256,))
    _check(load().wq_debug_mma_peak(kind, iters, blocks, _ptr(out), _stream()), "wq_debug_mma_peak")
    return out


def debug_w4a8_group_acc(x: torch.Tensor, packed4: torch.Tensor, scales: torch.Tensor, N: int, K: int,
                         acc: torch.Tensor | None = None) -> torch.Tensor:
    """The exact int32 group accumulators [M, N, K/128] of W4A8, from the
    kernel w4a8_gemm launches for the same shape (x is the bf16 activation,
    quantized per token exactly as w4a8_gemm does)."""
    M = x.shape[0]
    _need(x, "x", torch.bfloat16, (M, K))
    _need(packed4, "packed4", torch.int32, (N, packed_words_per_row(K, 4)))
    _need(scales, "scales", torch.bfloat16, (N, K // 128))
    if acc is None:
        acc = torch.empty((M, N, K // 128), dtype=torch.int32, device=x.device)
    _need(acc, "acc", torch.int32, (M, N, K // 128))
    scr = scratch(w4a8_scratch_bytes(M, K))
    _check(load().wq_debug_w4a8_group_acc(_ptr(x), M, _ptr(packed4), _ptr(scales), N, K, _ptr(acc), _ptr(scr),
                                          scr.numel() * scr.element_size(), _stream()),
           "wq_debug_w4a8_group_acc")
    return acc
