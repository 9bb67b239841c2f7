"""ctypes binding of libcpring.so: argument marshalling only.

Every computation runs in the library's CUDA kernels; torch supplies device
memory and streams.  If the library is missing the calls raise instead of
falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libcpring.so")

CP_OK = 0
STATUS_NAMES = {
    0: "CP_OK", -1: "CP_ERR_NULL", -2: "CP_ERR_SHAPE", -3: "CP_ERR_UNSUPPORTED",
    -4: "CP_ERR_ALIGN", -5: "CP_ERR_CUDA", -6: "CP_ERR_BUFFER", -7: "CP_ERR_DOC_OFFSETS",
    -8: "CP_ERR_TIMEOUT", -9: "CP_ERR_DEVICE", -10: "CP_ERR_SCRATCH",
    -11: "CP_ERR_CACHE",
}
STATUS_CODES = {v: k for k, v in STATUS_NAMES.items()}

_lib = None
_lock = threading.Lock()

_vp, _i, _i64, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
_SIGS = {
    "cp_ring_attn_fwd": [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp],
    "cp_ring_attn_fwd_noalloc": [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp],
    "cp_ring_attn_fwd_rank": [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp],
    "cp_ring_attn_fwd_f32": [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp],
    "cp_ring_step": [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _vp, _vp],
    "cp_ring_step_f32": [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _vp, _vp],
    "cp_lse_merge": [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp],
    "cp_lse_finalize": [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp],
    "cp_ring_schedule": [_i, _i, _i, _i, _i, _vp, _vp, _i64, ctypes.POINTER(_i64)],
    "cp_ring_traffic": [_i64, _i64, _i64, _i64, _i, _i, _i, ctypes.POINTER(_i64)],
    "cp_get_last_status": [_vp],
    "cp_status_string": [_i],
    "cp_launch_counts": [ctypes.POINTER(_i64)],
    "cp_test_set_wait_fault": [_i, _i64],
    "cp_ring_emulated_workspace_bytes": [_i, _i, _i, _i, _i],
    "cp_ulysses_workspace_bytes": [_i, _i, _i, _i, _i],
    "cp_ulysses_attn_fwd": [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _i64, _vp,
                            ctypes.POINTER(_i64)],
    "cp_ring_attn_fwd_emulated": [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp,
                                  _i64, _vp, _vp, ctypes.POINTER(_i64)],
    "cp_fp8_quantize": [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp],
    "cp_ring_attn_bwd_workspace_bytes": [_i, _i, _i, _i, _i],
    "cp_ring_schedule_device": [_i, _i, _i, _vp, _vp, _vp],
    "cp_ring_attn_bwd": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp,
                         _vp, _i64, _vp],
    "cp_ring_attn_fwd_fp8": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp,
                             _vp],
    "cp_ring_attn_fwd_host_workspace_bytes": [_i, _i, _i, _i, _i, _i],
    "cp_ring_attn_fwd_host": [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _i64,
                              _vp],
    "cp_ring_attn_fwd_host_f32": [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp,
                                  _i64, _vp],
    "cp_qk_norm_rope": [_vp, _vp, _vp, _vp, _vp, _vp, _f, _vp, _i, _i, _vp, _vp, _vp, _i, _i, _i,
                        _i, _i, _i, _vp],
    "cp_qk_norm_rope_bwd_workspace_bytes": [_i, _i, _i, _i, _i],
    "cp_qk_norm_rope_bwd": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _f, _vp, _i, _i, _vp, _vp, _vp,
                            _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _i64, _vp],
    "cp_paged_append": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _f, _vp, _i, _i,
                        _vp, _i, _i, _i, _vp],
    "cp_paged_attn_decode_workspace_bytes": [_i, _i, _i, _i, _i, _i],
    "cp_paged_attn_decode": [_vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _vp, _i64, _vp],
}


class PagedCacheStruct(ctypes.Structure):
    """cp_paged_cache of include/cpring.h."""
    _fields_ = [("k", _vp), ("v", _vp), ("k_strides", _i64 * 3), ("v_strides", _i64 * 3),
                ("k_descale", _vp), ("v_descale", _vp), ("page_table", _vp),
                ("table_stride", _i64), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("Hk", ctypes.c_int32), ("d", ctypes.c_int32), ("elem_bytes", ctypes.c_int32)]


class CpError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        self.name = STATUS_NAMES.get(status, str(status))
        super().__init__(f"{fn} failed: {self.name} ({status})")


def lib() -> ctypes.CDLL:
    """The loaded library (loaded once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -c 'import __graft_entry__ as g; g.build()'`")
            handle = ctypes.CDLL(LIB_PATH)
            for name, argtypes in _SIGS.items():
                fn = getattr(handle, name)
                fn.argtypes = argtypes
                if name == "cp_status_string":
                    fn.restype = ctypes.c_char_p
                elif name in ("cp_launch_counts", "cp_test_set_wait_fault"):
                    fn.restype = None
                elif name in ("cp_ring_emulated_workspace_bytes", "cp_ulysses_workspace_bytes",
                              "cp_ring_attn_bwd_workspace_bytes",
                              "cp_qk_norm_rope_bwd_workspace_bytes",
                              "cp_paged_attn_decode_workspace_bytes",
                              "cp_ring_attn_fwd_host_workspace_bytes"):
                    fn.restype = _i64
                else:
                    fn.restype = _i
            _lib = handle
    return _lib


def _check(fn: str, st: int) -> None:
    if st != CP_OK:
        raise CpError(fn, st)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape=None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def doc_offsets_tensor(doc_offsets, device) -> Optional[torch.Tensor]:
    """doc_offsets (list, numpy array or tensor) as a device int32 tensor."""
    if doc_offsets is None:
        return None
    if isinstance(doc_offsets, torch.Tensor):
        t = doc_offsets.to(device=device, dtype=torch.int32)
    else:
        t = torch.tensor([int(x) for x in doc_offsets], dtype=torch.int32, device=device)
    return t.contiguous()


# The calls around the attention are short enough on the device for their host side to
# count: the checks below read each property of a tensor once, and pointers travel as plain
# integers.
def _operand(t, name: str, dtype: torch.dtype, index: int, shape=None) -> int:
    """t's address, after checking its type, device, shape and that its last
    dimension is contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must live on cuda:{index}, got {t.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t.data_ptr()


def _dense(t, name: str, dtype: torch.dtype, index: int, shape=None) -> int:
    at = _operand(t, name, dtype, index, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return at


def _optional(t, name: str, dtype: torch.dtype, index: int, shape=None):
    return None if t is None else _dense(t, name, dtype, index, shape)


def _cuda_index(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must live on a CUDA device")
    return index


_Steps = _i64 * 3


def _steps(t):
    """The three leading strides of [a, b, c, d], None when contiguous.  The
    stride of a dimension of one entry is never used and passed as 0."""
    if t is None or t.is_contiguous():
        return None
    a, b, c, _ = t.stride()
    n = t.shape
    return _Steps(a if n[0] > 1 else 0, b if n[1] > 1 else 0, c if n[2] > 1 else 0)


def _call_on(name: str, index: int, stream, *args) -> None:
    """Run a library call with device `index` current, on `stream` or, if
    None, on that device's current stream."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    elif isinstance(stream, torch.cuda.Stream):
        if stream.device.index != index:
            raise ValueError(f"stream belongs to {stream.device}, the tensors to cuda:{index}")
        raw = stream.cuda_stream
    else:
        raw = int(stream)
    fn = getattr(_lib or lib(), name)
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            st = fn(*args, raw)
    if st != CP_OK:
        raise CpError(name, st)


# --------------------------------------------------------------------- C ABI
def cp_ring_attn_fwd(q, k, v, out, lse, n_shards: int, causal: bool = True,
                     doc_offsets: Optional[torch.Tensor] = None, stream=None) -> None:
    """bf16 fused forward; q, k, v, out [B,S,H,d] bf16, lse [B,H,S] fp32."""
    B, S, H, d = q.shape
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _need(t, n, torch.bfloat16, (B, S, H, d))
    _need(lse, "lse", torch.float32, (B, H, S))
    if doc_offsets is not None:
        _need(doc_offsets, "doc_offsets", torch.int32)
    _check("cp_ring_attn_fwd", lib().cp_ring_attn_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, S, H, d, int(n_shards),
        int(bool(causal)), _ptr(doc_offsets), _stream(stream)))


def cp_fp8_quantize(x, x8, descale, transpose: bool = False, stream=None) -> None:
    """Per-(b, h) E4M3 quantisation of x [B,S,H,d] bf16 into x8 (uint8,
    [B,S,H,d], or [B,H,d,S] with transpose) and descale [B,H] fp32."""
    B, S, H, d = x.shape
    _need(x, "x", torch.bfloat16)
    _need(x8, "x8", torch.uint8, (B, H, d, S) if transpose else (B, S, H, d))
    _need(descale, "descale", torch.float32, (B, H))
    _check("cp_fp8_quantize", lib().cp_fp8_quantize(
        _ptr(x), _ptr(x8), _ptr(descale), B, S, H, d, int(bool(transpose)), _stream(stream)))


def cp_ring_attn_fwd_fp8(q8, k8, v8t, q_descale, k_descale, v_descale, out, lse, n_shards: int,
                         causal: bool = True, doc_offsets: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    """FP8 fused forward: q8, k8 uint8 E4M3 [B,S,H,d], v8t uint8 E4M3
    [B,H,d,S], descales fp32 [B,H]; out [B,S,H,d] bf16, lse [B,H,S] fp32."""
    B, S, H, d = q8.shape
    _need(q8, "q8", torch.uint8, (B, S, H, d))
    _need(k8, "k8", torch.uint8, (B, S, H, d))
    _need(v8t, "v8t", torch.uint8, (B, H, d, S))
    for t, n in ((q_descale, "q_descale"), (k_descale, "k_descale"), (v_descale, "v_descale")):
        _need(t, n, torch.float32, (B, H))
    _need(out, "out", torch.bfloat16, (B, S, H, d))
    _need(lse, "lse", torch.float32, (B, H, S))
    if doc_offsets is not None:
        _need(doc_offsets, "doc_offsets", torch.int32)
    _check("cp_ring_attn_fwd_fp8", lib().cp_ring_attn_fwd_fp8(
        _ptr(q8), _ptr(k8), _ptr(v8t), _ptr(q_descale), _ptr(k_descale), _ptr(v_descale),
        _ptr(out), _ptr(lse), B, S, H, d, int(n_shards), int(bool(causal)), _ptr(doc_offsets),
        _stream(stream)))


def cp_ring_attn_bwd_workspace_bytes(B: int, S: int, H: int, d: int, n_shards: int) -> int:
    return int(lib().cp_ring_attn_bwd_workspace_bytes(B, S, H, d, n_shards))


def cp_ring_attn_bwd(q, k, v, out, lse, dout, dq, dk, dv, n_shards: int, causal: bool = True,
                     doc_offsets: Optional[torch.Tensor] = None, workspace=None,
                     stream=None) -> None:
    """bf16 backward: q, k, v, out, dout, dq, dk, dv [B,S,H,d] bf16, lse
    [B,H,S] fp32; workspace a uint8 device tensor of at least
    cp_ring_attn_bwd_workspace_bytes bytes (allocated here if None)."""
    B, S, H, d = q.shape
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout"), (dq, "dq"),
                 (dk, "dk"), (dv, "dv")):
        _need(t, n, torch.bfloat16, (B, S, H, d))
    _need(lse, "lse", torch.float32, (B, H, S))
    if doc_offsets is not None:
        _need(doc_offsets, "doc_offsets", torch.int32)
    need = cp_ring_attn_bwd_workspace_bytes(B, S, H, d, int(n_shards))
    if need < 0:
        raise CpError("cp_ring_attn_bwd_workspace_bytes", STATUS_CODES["CP_ERR_SHAPE"])
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check("cp_ring_attn_bwd", lib().cp_ring_attn_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
        _ptr(dv), B, S, H, d, int(n_shards), int(bool(causal)), _ptr(doc_offsets),
        _ptr(workspace), int(workspace.numel()), _stream(stream)))


def cp_ring_attn_fwd_rank(q, k, v, out, lse, n_shards: int, rank: int, causal: bool = True,
                          doc_offsets: Optional[torch.Tensor] = None, stream=None) -> None:
    """Rank `rank`'s part of the bf16 fused forward (its query shard's rows of
    out and lse); the tensors are the whole-sequence ones."""
    B, S, H, d = q.shape
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _need(t, n, torch.bfloat16, (B, S, H, d))
    _need(lse, "lse", torch.float32, (B, H, S))
    if doc_offsets is not None:
        _need(doc_offsets, "doc_offsets", torch.int32)
    _check("cp_ring_attn_fwd_rank", lib().cp_ring_attn_fwd_rank(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, S, H, d, int(n_shards), int(rank),
        int(bool(causal)), _ptr(doc_offsets), _stream(stream)))


def cp_ring_attn_fwd_host_workspace_bytes(B: int, S: int, H: int, d: int, n_shards: int,
                                          elem_bytes: int = 2) -> int:
    return int(lib().cp_ring_attn_fwd_host_workspace_bytes(B, S, H, d, n_shards, elem_bytes))


def _need_host(t: torch.Tensor, name: str, dtype: torch.dtype, shape) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.is_cuda:
        raise ValueError(f"{name} must live in host memory")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def cp_ring_attn_fwd_host(q_host, k_host, v_host, out_host, lse_host, n_shards: int,
                          causal: bool = True, doc_offsets: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """The fused forward from host tensors (bf16 or fp32 [B,S,H,d], lse fp32
    [B,H,S]; page-locked for overlap): asynchronous on `stream`, whose
    synchronisation completes out_host and lse_host.  workspace: a uint8
    device tensor of cp_ring_attn_fwd_host_workspace_bytes bytes."""
    B, S, H, d = q_host.shape
    dt = q_host.dtype
    if dt not in (torch.bfloat16, torch.float32):
        raise TypeError("q_host must be bf16 or fp32")
    for t, n in ((q_host, "q_host"), (k_host, "k_host"), (v_host, "v_host"),
                 (out_host, "out_host")):
        _need_host(t, n, dt, (B, S, H, d))
    _need_host(lse_host, "lse_host", torch.float32, (B, H, S))
    if doc_offsets is not None:
        _need(doc_offsets, "doc_offsets", torch.int32)
    if workspace is None:
        raise ValueError("workspace is required")
    _need(workspace, "workspace", torch.uint8)
    name = "cp_ring_attn_fwd_host" if dt == torch.bfloat16 else "cp_ring_attn_fwd_host_f32"
    _check(name, getattr(lib(), name)(
        _ptr(q_host), _ptr(k_host), _ptr(v_host), _ptr(out_host), _ptr(lse_host), B, S, H, d,
        int(n_shards), int(bool(causal)), _ptr(doc_offsets), _ptr(workspace),
        int(workspace.numel()), _stream(stream)))


def cp_ring_attn_fwd_noalloc(q, k, v, out, lse, n_shards: int, causal: bool = True,
                             doc_offsets: Optional[torch.Tensor] = None, stream=None) -> None:
    """cp_ring_attn_fwd without any device allocation by the library, for
    callers whose memory pool forbids it; at most 65,535 documents (more is
    reported as CP_ERR_SCRATCH by cp_get_last_status)."""
    B, S, H, d = q.shape
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _need(t, n, torch.bfloat16, (B, S, H, d))
    _need(lse, "lse", torch.float32, (B, H, S))
    if doc_offsets is not None:
        _need(doc_offsets, "doc_offsets", torch.int32)
    _check("cp_ring_attn_fwd_noalloc", lib().cp_ring_attn_fwd_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, S, H, d, int(n_shards),
        int(bool(causal)), _ptr(doc_offsets), _stream(stream)))


def cp_ring_attn_fwd_emulated(q, k, v, out, lse, n_shards: int, causal: bool = True,
                              workspace: Optional[torch.Tensor] = None, stream=None,
                              copy_stream=None, doc_offsets: Optional[torch.Tensor] = None):
    """The ring with explicit per-rank K/V buffers and copy-engine transfers
    (overlapped on copy_stream, or in order when copy_stream is None).
    Returns the bytes each rank received.  workspace: a uint8 device tensor
    of at least cp_ring_emulated_workspace_bytes(...) bytes (allocated here
    if None)."""
    B, S, H, d = q.shape
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _need(t, n, torch.bfloat16, (B, S, H, d))
    _need(lse, "lse", torch.float32, (B, H, S))
    if doc_offsets is not None:
        _need(doc_offsets, "doc_offsets", torch.int32)
    need = int(lib().cp_ring_emulated_workspace_bytes(B, S, H, d, int(n_shards)))
    if need < 0:
        raise CpError("cp_ring_emulated_workspace_bytes", STATUS_CODES["CP_ERR_SHAPE"])
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    recv = (ctypes.c_int64 * int(n_shards))()
    cs = None if copy_stream is None else _stream(copy_stream)
    _check("cp_ring_attn_fwd_emulated", lib().cp_ring_attn_fwd_emulated(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, S, H, d, int(n_shards),
        int(bool(causal)), _ptr(doc_offsets), _ptr(workspace), int(workspace.numel()),
        _stream(stream), cs, recv))
    return list(recv)


def cp_ulysses_attn_fwd(q, k, v, out, lse, n_shards: int, causal: bool = True,
                        doc_offsets: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> int:
    """All-to-all (Ulysses) form: head-split attention between two layout
    permutations.  Returns the bytes the two all-to-alls would move."""
    B, S, H, d = q.shape
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _need(t, n, torch.bfloat16, (B, S, H, d))
    _need(lse, "lse", torch.float32, (B, H, S))
    if doc_offsets is not None:
        _need(doc_offsets, "doc_offsets", torch.int32)
    need = int(lib().cp_ulysses_workspace_bytes(B, S, H, d, int(n_shards)))
    if need < 0:
        raise CpError("cp_ulysses_workspace_bytes", STATUS_CODES["CP_ERR_SHAPE"])
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    moved = ctypes.c_int64(0)
    _check("cp_ulysses_attn_fwd", lib().cp_ulysses_attn_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, S, H, d, int(n_shards),
        int(bool(causal)), _ptr(doc_offsets), _ptr(workspace), int(workspace.numel()),
        _stream(stream), ctypes.byref(moved)))
    return int(moved.value)


def cp_ulysses_workspace_bytes(B: int, S: int, H: int, d: int, n_shards: int) -> int:
    return int(lib().cp_ulysses_workspace_bytes(B, S, H, d, n_shards))


def cp_ring_emulated_workspace_bytes(B: int, S: int, H: int, d: int, n_shards: int) -> int:
    return int(lib().cp_ring_emulated_workspace_bytes(B, S, H, d, n_shards))


def cp_ring_attn_fwd_f32(q, k, v, out, lse, n_shards: int, causal: bool = True,
                         doc_offsets: Optional[torch.Tensor] = None, stream=None) -> None:
    """fp32 fused forward; q, k, v, out [B,S,H,d] fp32, lse [B,H,S] fp32."""
    B, S, H, d = q.shape
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _need(t, n, torch.float32, (B, S, H, d))
    _need(lse, "lse", torch.float32, (B, H, S))
    if doc_offsets is not None:
        _need(doc_offsets, "doc_offsets", torch.int32)
    _check("cp_ring_attn_fwd_f32", lib().cp_ring_attn_fwd_f32(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, S, H, d, int(n_shards),
        int(bool(causal)), _ptr(doc_offsets), _stream(stream)))


def cp_ring_step(q, k, v, o_part, m_part, l_part, n_shards: int, i: int, j: int,
                 causal: bool = True, doc_offsets: Optional[torch.Tensor] = None,
                 stream=None) -> None:
    """One partial step (i, j).  bf16 or fp32 q/k/v (dispatched on dtype);
    o_part [B,S/N,H,d] fp32, m_part and l_part [B,H,S/N] fp32."""
    B, S, H, d = q.shape
    L = S // int(n_shards) if n_shards else 0
    dt = q.dtype
    if dt not in (torch.bfloat16, torch.float32):
        raise TypeError("q must be bf16 or fp32")
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, dt, (B, S, H, d))
    _need(o_part, "o_part", torch.float32, (B, L, H, d))
    _need(m_part, "m_part", torch.float32, (B, H, L))
    _need(l_part, "l_part", torch.float32, (B, H, L))
    if doc_offsets is not None:
        _need(doc_offsets, "doc_offsets", torch.int32)
    name = "cp_ring_step" if dt == torch.bfloat16 else "cp_ring_step_f32"
    _check(name, getattr(lib(), name)(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o_part), _ptr(m_part), _ptr(l_part), B, S, H, d,
        int(n_shards), int(i), int(j), int(bool(causal)), _ptr(doc_offsets), _stream(stream)))


def cp_lse_merge(o_acc, m_acc, l_acc, o_part, m_part, l_part, stream=None) -> None:
    """In-place online merge of (o_part, m_part, l_part) into (o_acc, m_acc, l_acc)."""
    B, rows, H, d = o_acc.shape
    _need(o_acc, "o_acc", torch.float32)
    _need(o_part, "o_part", torch.float32, (B, rows, H, d))
    for t, n in ((m_acc, "m_acc"), (l_acc, "l_acc"), (m_part, "m_part"), (l_part, "l_part")):
        _need(t, n, torch.float32, (B, H, rows))
    _check("cp_lse_merge", lib().cp_lse_merge(
        _ptr(o_acc), _ptr(m_acc), _ptr(l_acc), _ptr(o_part), _ptr(m_part), _ptr(l_part),
        B, rows, H, d, _stream(stream)))


def cp_lse_finalize(o_acc, m_acc, l_acc, out, lse, stream=None) -> None:
    """out = o_acc / l_acc (bf16 or fp32 by out's dtype), lse = m + log(l)."""
    B, rows, H, d = o_acc.shape
    _need(o_acc, "o_acc", torch.float32)
    for t, n in ((m_acc, "m_acc"), (l_acc, "l_acc"), (lse, "lse")):
        _need(t, n, torch.float32, (B, H, rows))
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out must be bf16 or fp32")
    _need(out, "out", out.dtype, (B, rows, H, d))
    _check("cp_lse_finalize", lib().cp_lse_finalize(
        _ptr(o_acc), _ptr(m_acc), _ptr(l_acc), _ptr(out), _ptr(lse), B, rows, H, d,
        int(out.dtype == torch.bfloat16), _stream(stream)))


def cp_ring_schedule(S: int, n_shards: int, tile_q: int, tile_k: int, causal: bool = True,
                     doc_offsets: Optional[Sequence[int]] = None):
    """Host-side skip schedule: list of (q tile, kv tile) pairs."""
    L = lib()
    n = ctypes.c_int64(0)
    docs = None
    if doc_offsets is not None:
        arr = (ctypes.c_int32 * len(doc_offsets))(*[int(x) for x in doc_offsets])
        docs = ctypes.cast(arr, ctypes.c_void_p)
    _check("cp_ring_schedule", L.cp_ring_schedule(S, n_shards, tile_q, tile_k, int(bool(causal)),
                                                  docs, None, 0, ctypes.byref(n)))
    cnt = n.value
    buf = (ctypes.c_int32 * max(1, 2 * cnt))()
    _check("cp_ring_schedule", L.cp_ring_schedule(S, n_shards, tile_q, tile_k, int(bool(causal)),
                                                  docs, ctypes.cast(buf, ctypes.c_void_p), cnt,
                                                  ctypes.byref(n)))
    return [(buf[2 * x], buf[2 * x + 1]) for x in range(cnt)]


def cp_ring_schedule_device(S: int, n_shards: int, causal: bool = True,
                            doc_offsets: Optional[torch.Tensor] = None, device="cuda",
                            stream=None) -> torch.Tensor:
    """The fused kernel's key-tile range per 128-row query tile, computed on the
    device: int32 [n_tiles, 2] (first, last flat key tile)."""
    L = S // n_shards
    n_tiles = n_shards * ((L + 127) // 128)
    out = torch.full((n_tiles, 2), -7, dtype=torch.int32, device=device)
    if doc_offsets is not None:
        _need(doc_offsets, "doc_offsets", torch.int32)
    _check("cp_ring_schedule_device", lib().cp_ring_schedule_device(
        S, n_shards, int(bool(causal)), _ptr(doc_offsets), _ptr(out), _stream(stream)))
    return out


def cp_ring_traffic(B: int, S: int, H: int, d: int, dtype_bytes: int, n_shards: int,
                    causal: bool = False):
    """Per-rank send + receive bytes of the virtual ring."""
    out = (ctypes.c_int64 * n_shards)()
    _check("cp_ring_traffic", lib().cp_ring_traffic(B, S, H, d, dtype_bytes, n_shards,
                                                    int(bool(causal)), out))
    return list(out)


def cp_get_last_status(stream=None) -> int:
    """Synchronise the stream, read and clear the device error word."""
    return int(lib().cp_get_last_status(_stream(stream)))


def cp_status_string(status: int) -> str:
    return lib().cp_status_string(int(status)).decode()


def test_set_wait_fault(drop_first_k_tile: bool, wait_limit_ns: int = 0) -> None:
    """Test hook: make CTA 0 of later tensor-core launches skip its first K
    tile so that a bounded device wait runs out (see include/cpring.h)."""
    lib().cp_test_set_wait_fault(int(bool(drop_first_k_tile)), int(wait_limit_ns))


def launch_counts():
    """(tcgen05 attention, fp32 attention, merge/finalize, doc scan) launches so far."""
    buf = (ctypes.c_int64 * 4)()
    lib().cp_launch_counts(buf)
    return tuple(buf)


# ------------------------------------------------- norm, rotation, paged cache
def _rows4(t, name: str):
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise ValueError(f"{name} must be a tensor of four dimensions")
    return t.shape


def cp_qk_norm_rope(q, k, q_weight, k_weight, inv_freq, positions, q_out, k_out,
                    eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
    """Per-head RMS norm and rotation of q [B,S,Hq,d] and k [B,S,Hk,d] (bf16 or
    fp32, strided views allowed; k None: q only) into the contiguous q_out and
    k_out.  Weights fp32 [d] (None: not normed), inv_freq fp32 [rot_dim / 2]
    (None: not rotated), positions int32 [B,S] (None: the token's index)."""
    shape = _rows4(q, "q")
    B, S, Hq, d = shape
    dev, dt, f32 = _cuda_index(q, "q"), q.dtype, torch.float32
    if dt is not torch.bfloat16 and dt is not f32:
        raise TypeError("q must be bf16 or fp32")
    q_at, qo_at = _operand(q, "q", dt, dev), _dense(q_out, "q_out", dt, dev, shape)
    Hk, k_at, ko_at = 0, None, None
    if k is not None:
        Hk = _rows4(k, "k")[2]
        k_at = _operand(k, "k", dt, dev, (B, S, Hk, d))
        ko_at = _dense(k_out, "k_out", dt, dev, (B, S, Hk, d))
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    _call_on("cp_qk_norm_rope", dev, stream, q_at, _steps(q), k_at, _steps(k),
             _optional(q_weight, "q_weight", f32, dev, (d,)),
             _optional(k_weight, "k_weight", f32, dev, (d,)), eps,
             _optional(inv_freq, "inv_freq", f32, dev, (rot // 2,)), rot, bool(interleaved),
             _optional(positions, "positions", torch.int32, dev, (B, S)), qo_at, ko_at, B, S, Hq,
             Hk, d, dt is not f32)


def cp_qk_norm_rope_bwd_workspace_bytes(B: int, S: int, Hq: int, Hk: int, d: int) -> int:
    return int(lib().cp_qk_norm_rope_bwd_workspace_bytes(B, S, Hq, Hk, d))


def cp_qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, inv_freq, positions, dq, dk,
                        dq_weight, dk_weight, eps: float = 1e-6, interleaved: bool = False,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Backward of cp_qk_norm_rope: from dq_out, dk_out (contiguous) and the
    forward's inputs, writes dq, dk (the inputs' type, strided views allowed)
    and the weights' gradients (fp32 [d], or None).  workspace: a uint8 device
    tensor (allocated here if None)."""
    shape = _rows4(q, "q")
    B, S, Hq, d = shape
    dev, dt, f32 = _cuda_index(q, "q"), q.dtype, torch.float32
    if dt is not torch.bfloat16 and dt is not f32:
        raise TypeError("q must be bf16 or fp32")
    q_at, dq_at = _operand(q, "q", dt, dev), _operand(dq, "dq", dt, dev, shape)
    dqo_at = _dense(dq_out, "dq_out", dt, dev, shape)
    Hk, k_at, dk_at, dko_at, dk_steps = 0, None, None, None, None
    if k is not None:
        Hk = _rows4(k, "k")[2]
        k_at = _operand(k, "k", dt, dev, (B, S, Hk, d))
        dk_at = _operand(dk, "dk", dt, dev, (B, S, Hk, d))
        dko_at = _dense(dk_out, "dk_out", dt, dev, (B, S, Hk, d))
        dk_steps = _steps(dk)
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    if workspace is None:
        need = cp_qk_norm_rope_bwd_workspace_bytes(B, S, Hq, Hk, d)
        if need < 0:
            raise CpError("cp_qk_norm_rope_bwd_workspace_bytes", STATUS_CODES["CP_ERR_SHAPE"])
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _call_on("cp_qk_norm_rope_bwd", dev, stream, dqo_at, dko_at, q_at, _steps(q), k_at, _steps(k),
             _optional(q_weight, "q_weight", f32, dev, (d,)),
             _optional(k_weight, "k_weight", f32, dev, (d,)), eps,
             _optional(inv_freq, "inv_freq", f32, dev, (rot // 2,)), rot, bool(interleaved),
             _optional(positions, "positions", torch.int32, dev, (B, S)), dq_at, _steps(dq), dk_at,
             dk_steps, _optional(dq_weight, "dq_weight", f32, dev, (d,)),
             _optional(dk_weight, "dk_weight", f32, dev, (d,)), B, S, Hq, Hk, d, dt is not f32,
             _dense(workspace, "workspace", torch.uint8, dev), workspace.numel())


def _cache_struct(k_cache, v_cache, page_table, k_descale, v_descale, B: int,
                  dev: int) -> PagedCacheStruct:
    """The cp_paged_cache of caches [pages, page_size, Hk, d] (bf16, or uint8
    E4M3 codes with fp32 [Hk] descales) and an int32 table [B, max_pages]."""
    dt = k_cache.dtype if isinstance(k_cache, torch.Tensor) else None
    e4m3 = dt is torch.uint8
    if not e4m3 and dt is not torch.bfloat16:
        raise TypeError("k_cache must be bf16 or uint8 (E4M3 codes)")
    shape = _rows4(k_cache, "k_cache")
    n_pages, page_size, Hk, d = shape
    k_at = _operand(k_cache, "k_cache", dt, dev)
    v_at = _operand(v_cache, "v_cache", dt, dev, shape)
    table_at = _operand(page_table, "page_table", torch.int32, dev)
    if page_table.dim() != 2:
        raise ValueError("page_table must have two dimensions")
    rows, max_pages = page_table.shape
    if rows != B:
        raise ValueError(f"page_table must have {B} rows, got {rows}")
    if e4m3:
        kd_at = _dense(k_descale, "k_descale", torch.float32, dev, (Hk,))
        vd_at = _dense(v_descale, "v_descale", torch.float32, dev, (Hk,))
    elif k_descale is None and v_descale is None:
        kd_at = vd_at = None
    else:
        raise ValueError("k_descale and v_descale go with an E4M3 cache")
    ks = v_s = _Steps(page_size * Hk * d, Hk * d, d)
    if not k_cache.is_contiguous():
        ks = _steps(k_cache)
    if not v_cache.is_contiguous():
        v_s = _steps(v_cache)
    return PagedCacheStruct(k_at, v_at, ks, v_s, kd_at, vd_at, table_at,
                            page_table.stride(0) if rows > 1 else max_pages, n_pages, page_size,
                            max_pages, Hk, d, 1 if e4m3 else 2)


def cp_paged_append(q, k, v, k_cache, v_cache, page_table, cache_lens, new_lens, q_weight,
                    k_weight, inv_freq, q_out, eps: float = 1e-6, interleaved: bool = False,
                    k_descale=None, v_descale=None, stream=None) -> None:
    """Norm, rotate and append k, v [B,S,Hk,d] bf16 (strided views allowed) to
    the paged caches [pages, page_size, Hk, d] at positions cache_lens[b] + s
    (int32 [B]), for s < new_lens[b] (int32 [B], None: all S); q [B,S,Hq,d]
    (None: keys and values only) is normed and rotated into q_out."""
    B, S, Hk, d = _rows4(k, "k")
    dev, bf16, i32, f32 = _cuda_index(k, "k"), torch.bfloat16, torch.int32, torch.float32
    cache = _cache_struct(k_cache, v_cache, page_table, k_descale, v_descale, B, dev)
    shape = (B, S, cache.Hk, cache.d)
    k_at, v_at = _operand(k, "k", bf16, dev, shape), _operand(v, "v", bf16, dev, shape)
    Hq, q_at, qo_at = 0, None, None
    if q is not None:
        Hq = _rows4(q, "q")[2]
        q_at = _operand(q, "q", bf16, dev, (B, S, Hq, d))
        qo_at = _dense(q_out, "q_out", bf16, dev, (B, S, Hq, d))
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    _call_on("cp_paged_append", dev, stream, ctypes.byref(cache), q_at, _steps(q), k_at, _steps(k),
             v_at, _steps(v), _dense(cache_lens, "cache_lens", i32, dev, (B,)),
             _optional(new_lens, "new_lens", i32, dev, (B,)),
             _optional(q_weight, "q_weight", f32, dev, (d,)),
             _optional(k_weight, "k_weight", f32, dev, (d,)), eps,
             _optional(inv_freq, "inv_freq", f32, dev, (rot // 2,)), rot, bool(interleaved), qo_at,
             B, S, Hq)


def cp_paged_attn_decode_workspace_bytes(B: int, n_q: int, Hq: int, Hk: int, d: int,
                                         prefix_len: int = 0) -> int:
    return int(lib().cp_paged_attn_decode_workspace_bytes(B, n_q, Hq, Hk, d, prefix_len))


def cp_paged_attn_decode(q, k_cache, v_cache, page_table, seq_lens, out, lse, prefix_pages=None,
                         prefix_len: int = 0, k_descale=None, v_descale=None,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Decode attention of q [B,n_q,Hq,d] bf16 (strided views allowed), the
    last n_q tokens of each sequence of seq_lens (int32 [B], 0 = unused row),
    over the paged caches of cp_paged_append; the keys of positions below
    prefix_len are read through prefix_pages (int32) once for the whole batch.
    out [B,n_q,Hq,d] bf16, lse [B,Hq,n_q] fp32; workspace a uint8 device
    tensor (allocated here if None)."""
    B, n_q, Hq, d = _rows4(q, "q")
    dev, bf16, i32 = _cuda_index(q, "q"), torch.bfloat16, torch.int32
    cache = _cache_struct(k_cache, v_cache, page_table, k_descale, v_descale, B, dev)
    shape = (B, n_q, Hq, cache.d)
    q_at, out_at = _operand(q, "q", bf16, dev, shape), _dense(out, "out", bf16, dev, shape)
    lse_at = _dense(lse, "lse", torch.float32, dev, (B, Hq, n_q))
    prefix_len, pages_at = int(prefix_len), None
    if prefix_pages is not None:
        pages_at = _dense(prefix_pages, "prefix_pages", i32, dev, (prefix_pages.numel(),))
        if prefix_pages.numel() * cache.page_size < prefix_len:
            raise ValueError("prefix_pages holds fewer tokens than prefix_len")
    if workspace is None:
        need = cp_paged_attn_decode_workspace_bytes(B, n_q, Hq, cache.Hk, d, prefix_len)
        if need < 0:
            raise CpError("cp_paged_attn_decode_workspace_bytes", STATUS_CODES["CP_ERR_SHAPE"])
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _call_on("cp_paged_attn_decode", dev, stream, ctypes.byref(cache), q_at, _steps(q),
             _dense(seq_lens, "seq_lens", i32, dev, (B,)), pages_at, prefix_len, out_at, lse_at, B,
             n_q, Hq, _dense(workspace, "workspace", torch.uint8, dev), workspace.numel())
