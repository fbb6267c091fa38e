"""ctypes binding of libsparse_mla.so (argument marshalling only)."""

import contextlib
import ctypes
import functools
from pathlib import Path
from typing import Optional, Tuple

import torch

_LIB_PATH = Path(__file__).resolve().parent / "libsparse_mla.so"
_lib = None

KV_FORMATS = {"bf16": 0, "fp8": 1}
D_QK, D_V, FP8_ROW_BYTES = 576, 512, 656

_STATUS = {0: "SMLA_OK", 1: "SMLA_ERR_INVALID_ARG", 2: "SMLA_ERR_UNSUPPORTED",
           3: "SMLA_ERR_CUDA", 4: "SMLA_ERR_TIMEOUT", 5: "SMLA_ERR_INDEX_RANGE"}
SMLA_ERR_INDEX_RANGE = 5

EXPORTED = ("sparse_mla_fwd", "sparse_mla_fwd_ex", "sparse_mla_fwd_checked", "sparse_mla_fwd_noalloc",
            "sparse_mla_fwd_host", "sparse_mla_fwd_host_packed", "sparse_mla_host_io_layout",
            "sparse_mla_host_workspace_bytes", "sparse_mla_merge",
            "sparse_mla_v_up", "sparse_mla_topk", "sparse_mla_scatter_mask", "sparse_mla_masked_mha",
            "sparse_mla_append", "sparse_mla_q_up", "sparse_mla_prefix", "sparse_mla_prefix_workspace_bytes",
            "sparse_mla_tree", "sparse_mla_tree_workspace_bytes",
            "sparse_mla_weights", "sparse_mla_evict",
            "sparse_mla_sync_status",
            "sparse_mla_launch_info", "sparse_mla_last_error", "sparse_mla_version")


class SparseMLAError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        super().__init__(f"{_STATUS.get(status, status)}: {message}")


def lib_path() -> Path:
    return _LIB_PATH


def library() -> ctypes.CDLL:
    """Load libsparse_mla.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not _LIB_PATH.exists():
        raise ImportError(f"{_LIB_PATH} is missing: build it with "
                          "`python -m token_sparse_mla_gb300.build` (nvcc, sm_103a)")
    lib = ctypes.CDLL(str(_LIB_PATH))
    vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                             ctypes.c_size_t)
    lib.sparse_mla_fwd.restype = ctypes.c_int
    lib.sparse_mla_fwd.argtypes = [vp, vp, vp, i32, i32, i32, i64, i32, f32, vp, vp, vp]
    lib.sparse_mla_fwd_ex.restype = ctypes.c_int
    lib.sparse_mla_fwd_ex.argtypes = [vp, vp, vp, i32, i32, i32, i64, i32, f32, vp, vp, i32, vp]
    lib.sparse_mla_fwd_checked.restype = ctypes.c_int
    lib.sparse_mla_fwd_checked.argtypes = [vp, vp, vp, i32, i32, i32, i64, i32, f32, vp, vp, i32, vp]
    lib.sparse_mla_fwd_noalloc.restype = ctypes.c_int
    lib.sparse_mla_fwd_noalloc.argtypes = [vp, vp, vp, i32, i32, i32, i64, i32, f32, vp, vp, i32, vp]
    lib.sparse_mla_topk.restype = ctypes.c_int
    lib.sparse_mla_topk.argtypes = [vp, i32, i64, vp, i32, vp, vp, vp]
    lib.sparse_mla_v_up.restype = ctypes.c_int
    lib.sparse_mla_v_up.argtypes = [vp, vp, i32, i32, i32, vp, vp]
    lib.sparse_mla_merge.restype = ctypes.c_int
    lib.sparse_mla_merge.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp]
    lib.sparse_mla_host_workspace_bytes.restype = sz
    lib.sparse_mla_host_workspace_bytes.argtypes = [i32, i32, i32]
    lib.sparse_mla_fwd_host.restype = ctypes.c_int
    lib.sparse_mla_fwd_host.argtypes = [vp, vp, vp, i32, i32, i32, i64, i32, f32, vp, vp, vp, sz, vp]
    lib.sparse_mla_scatter_mask.restype = ctypes.c_int
    lib.sparse_mla_scatter_mask.argtypes = [vp, i32, i32, i64, vp, vp]
    lib.sparse_mla_masked_mha.restype = ctypes.c_int
    lib.sparse_mla_masked_mha.argtypes = [vp, vp, vp, vp, i32, i64, i32, i32, i32, f32, vp, vp, vp]
    lib.sparse_mla_append.restype = ctypes.c_int
    lib.sparse_mla_append.argtypes = [vp, i64, vp, vp, i32, vp, i32, i32, vp, f32, vp, i64, i32, vp]
    lib.sparse_mla_q_up.restype = ctypes.c_int
    lib.sparse_mla_q_up.argtypes = [vp, vp, vp, i32, i32, i32, vp, i32, i32, vp, vp]
    lib.sparse_mla_prefix_workspace_bytes.restype = sz
    lib.sparse_mla_prefix_workspace_bytes.argtypes = [i32, i32, i64, i32]
    lib.sparse_mla_prefix.restype = ctypes.c_int
    lib.sparse_mla_prefix.argtypes = [vp, vp, vp, i32, i32, i64, i64, i32, f32, vp, vp, vp, sz, vp]
    lib.sparse_mla_tree_workspace_bytes.restype = sz
    lib.sparse_mla_tree_workspace_bytes.argtypes = [i32, i32, i32]
    lib.sparse_mla_tree.restype = ctypes.c_int
    lib.sparse_mla_tree.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i64, i32, f32, vp, vp, vp, sz, vp]
    lib.sparse_mla_weights.restype = ctypes.c_int
    lib.sparse_mla_weights.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, f32, i32, i32, i32, i32, i32, i64, i32, f32, vp, vp]
    lib.sparse_mla_evict.restype = ctypes.c_int
    lib.sparse_mla_evict.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i64, i32, vp, vp, vp, vp]
    lib.sparse_mla_host_io_layout.restype = ctypes.c_int
    lib.sparse_mla_host_io_layout.argtypes = [i32, i32, i32, vp, vp, vp, vp]
    lib.sparse_mla_fwd_host_packed.restype = ctypes.c_int
    lib.sparse_mla_fwd_host_packed.argtypes = [vp, vp, i32, i32, i32, i64, i32, f32, vp, vp, sz, vp]
    lib.sparse_mla_sync_status.restype = ctypes.c_int
    lib.sparse_mla_sync_status.argtypes = [vp]
    lib.sparse_mla_launch_info.restype = ctypes.c_int
    lib.sparse_mla_launch_info.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp]
    lib.sparse_mla_last_error.restype = ctypes.c_char_p
    lib.sparse_mla_last_error.argtypes = []
    lib.sparse_mla_version.restype = ctypes.c_int32
    lib.sparse_mla_version.argtypes = []
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != 0:
        msg = library().sparse_mla_last_error().decode(errors="replace")
        raise SparseMLAError(status, msg)


def _device_of(tensors) -> torch.device:
    """The one CUDA device that all (name, tensor) pairs live on; raises if there is none."""
    dev = None
    for name, t in tensors:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other tensors on {dev}")
    return dev


def _on(dev: torch.device):
    """Context that makes `dev` the current device: a no-op when it already is (entering
    torch.cuda.device costs several microseconds a call, a sizeable share of a decode step)."""
    return contextlib.nullcontext() if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _stream_handle(stream, device: Optional[torch.device] = None) -> Optional[int]:
    """Raw handle of `stream` (default: the current stream of `device`, else of the current
    device).  A stream object must belong to `device`; a raw int handle is passed as is."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    if isinstance(stream, int):
        return stream
    if device is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return stream.cuda_stream


def _current_handle(dev: torch.device) -> int:
    """Raw handle of torch's current stream on dev (a stream object costs 2 us to make)."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _empty(shape, dtype: torch.dtype, dev: torch.device, stream, result: bool = True) -> torch.Tensor:
    """An uninitialised tensor that a call on `stream` (None: the current one) writes.  A block of torch's
    allocator may still be in use by work pending on the stream that it was allocated for, and a freed one
    goes to the next request on that stream: so the tensor is allocated for the call's stream, and a
    result's use by the caller's current stream is recorded (scratch is used by the call alone)."""
    if stream is not None:
        handle = _stream_handle(stream, dev) or 0
        if handle != _current_handle(dev):
            # (1 is the legacy default stream's other name)
            with torch.cuda.stream(torch.cuda.ExternalStream(0 if handle == 1 else handle, device=dev)):
                t = torch.empty(shape, dtype=dtype, device=dev)
            if result:
                t.record_stream(torch.cuda.current_stream(dev))
            return t
    return torch.empty(shape, dtype=dtype, device=dev)


def version() -> int:
    return int(library().sparse_mla_version())


def _dims(q: torch.Tensor, kv_cache: torch.Tensor, indices: torch.Tensor, kv_format: str):
    if q.dim() != 3 or q.shape[2] != D_QK or q.dtype != torch.bfloat16:
        raise ValueError(f"q must be [T, h, 576] bf16, got {tuple(q.shape)} {q.dtype}")
    T, h = int(q.shape[0]), int(q.shape[1])
    if indices.dim() != 2 or indices.shape[0] != T or indices.dtype != torch.int32:
        raise ValueError(f"indices must be [T, topk] int32, got {tuple(indices.shape)} {indices.dtype}")
    if kv_format not in KV_FORMATS:
        raise ValueError(f"kv_format must be one of {sorted(KV_FORMATS)}")
    if kv_format == "bf16":
        if kv_cache.dim() != 2 or kv_cache.shape[1] != D_QK or kv_cache.dtype != torch.bfloat16:
            raise ValueError(f"bf16 kv_cache must be [num_slots, 576] bf16, got "
                             f"{tuple(kv_cache.shape)} {kv_cache.dtype}")
    else:
        if kv_cache.dim() != 2 or kv_cache.shape[1] != FP8_ROW_BYTES or kv_cache.dtype != torch.uint8:
            raise ValueError(f"fp8 kv_cache must be [num_slots, 656] uint8, got "
                             f"{tuple(kv_cache.shape)} {kv_cache.dtype}")
    for name, t in (("q", q), ("kv_cache", kv_cache), ("indices", indices)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return T, h, int(indices.shape[1]), int(kv_cache.shape[0])


def sparse_mla_fwd(q: torch.Tensor, kv_cache: torch.Tensor, indices: torch.Tensor,
                   scale: Optional[float] = None, *, out: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, kv_format: str = "bf16",
                   splits: int = 0, checked: bool = False,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Token-sparse MLA forward on the GPU (see include/sparse_mla.h).

    scale defaults to 576 ** -0.5.  out / lse may be passed in (caller-owned
    buffers, [T, h, 512] bf16 and [T, h] fp32); otherwise they are allocated
    here.  splits = 0 lets the library choose how many CTAs share a token's
    list.  checked = True runs sparse_mla_fwd_checked: the same outputs, and list
    entries other than -1 outside [0, num_slots) make the next sync_status()
    raise SMLA_ERR_INDEX_RANGE.  Runs asynchronously on `stream` (default:
    torch's current stream).
    """
    T, h, topk, num_slots = _dims(q, kv_cache, indices, kv_format)
    dev = _device_of((("q", q), ("kv_cache", kv_cache), ("indices", indices)))
    if scale is None:
        scale = D_QK ** -0.5
    if out is None:
        out = _empty((T, h, D_V), torch.bfloat16, dev, stream)
    if lse is None:
        lse = _empty((T, h), torch.float32, dev, stream)
    if out.shape != (T, h, D_V) or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous [T, h, 512] bf16 tensor")
    if lse.shape != (T, h) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous [T, h] fp32 tensor")
    _device_of((("q", q), ("out", out), ("lse", lse)))
    with _on(dev):
        lib = library()
        fn = lib.sparse_mla_fwd_checked if checked else lib.sparse_mla_fwd_ex
        st = fn(
            q.data_ptr(), kv_cache.data_ptr(), indices.data_ptr(), T, h, topk, num_slots,
            KV_FORMATS[kv_format], float(scale), out.data_ptr(), lse.data_ptr(), int(splits),
            _stream_handle(stream, dev))
    _check(st)
    return out, lse


def sparse_mla_fwd_noalloc(q: torch.Tensor, kv_cache: torch.Tensor, indices: torch.Tensor,
                           scale: Optional[float] = None, *, out: torch.Tensor, lse: torch.Tensor,
                           kv_format: str = "bf16", splits: int = 0, stream=None) -> None:
    """sparse_mla_fwd with the library's static merge scratch: nothing is allocated, so out and
    lse are required (see include/sparse_mla.h for the rules on first call and streams)."""
    T, h, topk, num_slots = _dims(q, kv_cache, indices, kv_format)
    dev = _device_of((("q", q), ("kv_cache", kv_cache), ("indices", indices), ("out", out),
                      ("lse", lse)))
    if scale is None:
        scale = D_QK ** -0.5
    if out.shape != (T, h, D_V) or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous [T, h, 512] bf16 tensor")
    if lse.shape != (T, h) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous [T, h] fp32 tensor")
    with _on(dev):
        st = library().sparse_mla_fwd_noalloc(
            q.data_ptr(), kv_cache.data_ptr(), indices.data_ptr(), T, h, topk, num_slots,
            KV_FORMATS[kv_format], float(scale), out.data_ptr(), lse.data_ptr(), int(splits),
            _stream_handle(stream, dev))
    _check(st)


def sparse_mla_merge(o_parts: torch.Tensor, lse_parts: torch.Tensor, *,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Merge the partial results of split token lists (the DCP merge; include/sparse_mla.h).

    o_parts [n, T, h, 512] bf16 and lse_parts [n, T, h] fp32 are what sparse_mla_fwd returned
    for each of the n parts (LSE -inf = empty part); returns out [T, h, 512] bf16 and
    lse [T, h] fp32 of the whole lists.
    """
    if o_parts.dim() != 4 or o_parts.shape[-1] != D_V or o_parts.dtype != torch.bfloat16:
        raise ValueError("o_parts must be [n, T, h, 512] bf16")
    n, T, h = int(o_parts.shape[0]), int(o_parts.shape[1]), int(o_parts.shape[2])
    if lse_parts.shape != (n, T, h) or lse_parts.dtype != torch.float32:
        raise ValueError("lse_parts must be [n, T, h] fp32")
    dev = _device_of((("o_parts", o_parts), ("lse_parts", lse_parts)))
    for name, t in (("o_parts", o_parts), ("lse_parts", lse_parts)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if out is None:
        out = _empty((T, h, D_V), torch.bfloat16, dev, stream)
    if lse is None:
        lse = _empty((T, h), torch.float32, dev, stream)
    if out.shape != (T, h, D_V) or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous [T, h, 512] bf16 tensor")
    if lse.shape != (T, h) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous [T, h] fp32 tensor")
    _device_of((("o_parts", o_parts), ("out", out), ("lse", lse)))
    with _on(dev):
        st = library().sparse_mla_merge(o_parts.data_ptr(), lse_parts.data_ptr(), n, T, h,
                                        out.data_ptr(), lse.data_ptr(), _stream_handle(stream, dev))
    _check(st)
    return out, lse


def sparse_mla_v_up(o: torch.Tensor, w: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """The v_up projection of the attention output on the tensor cores (include/sparse_mla.h):
    y[t, h, n] = sum_k o[t, h, k] * w[h, n, k], o [T, h, 512] bf16, w [h, v, 512] bf16
    (v = 128 or 256); returns y [T, h, v] bf16."""
    if o.dim() != 3 or o.shape[-1] != D_V or o.dtype != torch.bfloat16:
        raise ValueError("o must be [T, h, 512] bf16")
    T, h = int(o.shape[0]), int(o.shape[1])
    if w.dim() != 3 or w.shape[0] != h or w.shape[2] != D_V or w.dtype != torch.bfloat16:
        raise ValueError("w must be [h, v, 512] bf16")
    v = int(w.shape[1])
    dev = _device_of((("o", o), ("w", w)))
    for name, t in (("o", o), ("w", w)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if out is None:
        out = _empty((T, h, v), torch.bfloat16, dev, stream)
    if out.shape != (T, h, v) or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous [T, h, v] bf16 tensor")
    _device_of((("o", o), ("out", out)))
    with _on(dev):
        st = library().sparse_mla_v_up(o.data_ptr(), w.data_ptr(), T, h, v, out.data_ptr(),
                                       _stream_handle(stream, dev))
    _check(st)
    return out


def sparse_mla_topk(scores: torch.Tensor, lengths: torch.Tensor, topk: int, *,
                    block_table: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """Index lists from per-position scores (include/sparse_mla.h): the top `topk` positions of
    scores[t, :lengths[t]] (ties to the lower position), ascending, mapped through block_table
    (64-slot blocks) when given, -1 padded.  scores [T, S] fp32, lengths [T] int32."""
    if scores.dim() != 2 or scores.dtype != torch.float32:
        raise ValueError("scores must be [T, S] fp32")
    T, S = int(scores.shape[0]), int(scores.shape[1])
    if lengths.shape != (T,) or lengths.dtype != torch.int32:
        raise ValueError("lengths must be [T] int32")
    tensors = [("scores", scores), ("lengths", lengths)]
    if block_table is not None:
        if block_table.dim() != 1 or block_table.dtype != torch.int32 or block_table.numel() * 64 < S:
            raise ValueError("block_table must be [ceil(S / 64)] int32")
        tensors.append(("block_table", block_table))
    dev = _device_of(tensors)
    for name, t in tensors:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if out is None:
        out = _empty((T, topk), torch.int32, dev, stream)
    if out.shape != (T, topk) or out.dtype != torch.int32 or not out.is_contiguous():
        raise ValueError("out must be a contiguous [T, topk] int32 tensor")
    _device_of((("scores", scores), ("out", out)))
    with _on(dev):
        st = library().sparse_mla_topk(scores.data_ptr(), T, S, lengths.data_ptr(), int(topk),
                                       None if block_table is None else block_table.data_ptr(),
                                       out.data_ptr(), _stream_handle(stream, dev))
    _check(st)
    return out


def sparse_mla_scatter_mask(indices: torch.Tensor, S: int, *, out: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """The lists of one request as a bit mask (include/sparse_mla.h): indices [T, topk] int32
    positions; returns mask [T, ceil(S / 32)] int32 whose bit s % 32 of word s / 32 is set iff s
    is listed (the words are uint32 bit patterns, held in an int32 tensor)."""
    if indices.dim() != 2 or indices.dtype != torch.int32:
        raise ValueError("indices must be [T, topk] int32")
    T, topk = int(indices.shape[0]), int(indices.shape[1])
    W = (int(S) + 31) // 32
    dev = _device_of((("indices", indices),))
    if not indices.is_contiguous():
        raise ValueError("indices must be contiguous")
    if out is None:
        out = _empty((T, W), torch.int32, dev, stream)
    if out.shape != (T, W) or out.dtype != torch.int32 or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous [T, {W}] int32 tensor")
    _device_of((("indices", indices), ("out", out)))
    with _on(dev):
        st = library().sparse_mla_scatter_mask(indices.data_ptr(), T, topk, int(S), out.data_ptr(),
                                               _stream_handle(stream, dev))
    _check(st)
    return out


def sparse_mla_masked_mha(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, mask: torch.Tensor,
                          scale: float, *, out: Optional[torch.Tensor] = None,
                          lse: Optional[torch.Tensor] = None,
                          stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Masked dense MHA (include/sparse_mla.h): q [T, h, dqk], k [S, h, dqk], v [S, h, dv] bf16,
    mask [T, ceil(S / 32)] int32 bit words; returns out [T, h, dv] bf16 and lse [T, h] fp32."""
    if q.dim() != 3 or q.dtype != torch.bfloat16:
        raise ValueError("q must be [T, h, dqk] bf16")
    T, h, dqk = (int(x) for x in q.shape)
    if k.dim() != 3 or k.dtype != torch.bfloat16 or k.shape[1] != h or k.shape[2] != dqk:
        raise ValueError("k must be [S, h, dqk] bf16")
    S = int(k.shape[0])
    if v.dim() != 3 or v.dtype != torch.bfloat16 or v.shape[0] != S or v.shape[1] != h:
        raise ValueError("v must be [S, h, dv] bf16")
    dv = int(v.shape[2])
    W = (S + 31) // 32
    if mask.shape != (T, W) or mask.dtype != torch.int32:
        raise ValueError(f"mask must be [T, {W}] int32")
    tensors = (("q", q), ("k", k), ("v", v), ("mask", mask))
    dev = _device_of(tensors)
    for name, t in tensors:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if out is None:
        out = _empty((T, h, dv), torch.bfloat16, dev, stream)
    if lse is None:
        lse = _empty((T, h), torch.float32, dev, stream)
    if out.shape != (T, h, dv) or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous [T, h, {dv}] bf16 tensor")
    if lse.shape != (T, h) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous [T, h] fp32 tensor")
    _device_of((("q", q), ("out", out), ("lse", lse)))
    with _on(dev):
        st = library().sparse_mla_masked_mha(q.data_ptr(), k.data_ptr(), v.data_ptr(), mask.data_ptr(), T, S, h,
                                             dqk, dv, float(scale), out.data_ptr(), lse.data_ptr(),
                                             _stream_handle(stream, dev))
    _check(st)
    return out, lse


# ---- append, q_up and prefix.  A decode step makes these calls once per layer, so what they cost on the
# host counts: a call of theirs reads each tensor's attributes once, takes the raw stream handle and
# enters no context when the device is already current.

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _call(dev: torch.device, stream, fn, *args) -> None:
    """fn(*args, stream handle) with dev current; raises on a status other than OK."""
    handle = _current_handle(dev) if stream is None else _stream_handle(stream, dev)
    if torch.cuda.current_device() == dev.index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st != 0:
        _check(st)


def _given(name: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype, dev: torch.device) -> torch.Tensor:
    """A tensor that the caller passed, checked."""
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} {dtype} tensor")
    if t.device != dev:
        _apart(dev, **{name: t})
    return t


def _apart(dev: torch.device, **tensors) -> None:
    """Names the first tensor that is not on dev."""
    for name, t in tensors.items():
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other tensors on {dev}")


def _cuda_device(name: str, t: torch.Tensor) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    return t.device


def _positions_and_table(T: int, positions: torch.Tensor, cos_sin: torch.Tensor) -> int:
    if positions.shape != (T,) or positions.dtype != _I32 or not positions.is_contiguous():
        raise ValueError(f"positions must be a contiguous [{T}] int32 tensor")
    if cos_sin.dim() != 2 or cos_sin.shape[1] != D_QK - D_V or cos_sin.dtype != _F32 or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be a contiguous [max_pos, 64] fp32 tensor")
    return cos_sin.shape[0]


def _cache_rows(kv_cache: torch.Tensor, kv_format: str) -> int:
    """num_slots of a cache tensor of the given format."""
    if kv_format not in KV_FORMATS:
        raise ValueError(f"kv_format must be one of {sorted(KV_FORMATS)}")
    row, dtype = (D_QK, _BF16) if kv_format == "bf16" else (FP8_ROW_BYTES, _U8)
    if kv_cache.dim() != 2 or kv_cache.shape[1] != row or kv_cache.dtype != dtype or not kv_cache.is_contiguous():
        raise ValueError(f"{kv_format} kv_cache must be a contiguous [num_slots, {row}] {dtype} tensor, got "
                         f"{tuple(kv_cache.shape)} {kv_cache.dtype}")
    return kv_cache.shape[0]


def sparse_mla_append(kv: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor, kv_cache: torch.Tensor,
                      cos_sin: torch.Tensor, *, norm_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                      interleaved: bool = True, kv_format: str = "bf16", stream=None) -> torch.Tensor:
    """Write new tokens' rows into the paged latent cache (include/sparse_mla.h): the latent (through
    its RMS norm when norm_weight is given), the rope dims rotated by their position, as bf16 or fp8
    rows.  Returns kv_cache, written in place.

    kv [T, 576] bf16, 512 latent then 64 rope dims; rows may lie apart (a slice of a fused
    projection's output) as long as each is contiguous.  positions and slots [T] int32, slot -1 =
    write nothing.  cos_sin [max_pos, 64] fp32, 32 cosines then 32 sines a row.  The slots other than
    -1 must be distinct.  A slot or position out of range writes nothing and makes the next
    sync_status() raise SMLA_ERR_INDEX_RANGE.
    """
    if kv.dim() != 2 or kv.shape[1] != D_QK or kv.dtype != _BF16:
        raise ValueError(f"kv must be [T, 576] bf16, got {tuple(kv.shape)} {kv.dtype}")
    T = kv.shape[0]
    row_stride, inner = kv.stride()
    if T <= 1:
        row_stride = D_QK
    if inner != 1 or row_stride < D_QK or row_stride % 8:
        raise ValueError(f"kv rows must be contiguous and a multiple of 8 elements (>= 576) apart, "
                         f"got strides {tuple(kv.stride())}")
    if slots.shape != (T,) or slots.dtype != _I32 or not slots.is_contiguous():
        raise ValueError(f"slots must be a contiguous [{T}] int32 tensor")
    max_pos = _positions_and_table(T, positions, cos_sin)
    num_slots = _cache_rows(kv_cache, kv_format)
    dev = _cuda_device("kv", kv)
    if not dev == positions.device == slots.device == kv_cache.device == cos_sin.device:
        _apart(dev, positions=positions, slots=slots, kv_cache=kv_cache, cos_sin=cos_sin)
    weight = None
    if norm_weight is not None:
        if norm_weight.shape != (D_V,) or norm_weight.dtype != _BF16 or not norm_weight.is_contiguous():
            raise ValueError("norm_weight must be a contiguous [512] bf16 tensor")
        if norm_weight.device != dev:
            _apart(dev, norm_weight=norm_weight)
        weight = norm_weight.data_ptr()
    _call(dev, stream, library().sparse_mla_append, kv.data_ptr(), row_stride, positions.data_ptr(), slots.data_ptr(),
          T, cos_sin.data_ptr(), max_pos, 1 if interleaved else 0, weight, float(eps), kv_cache.data_ptr(), num_slots,
          KV_FORMATS[kv_format])
    return kv_cache


def sparse_mla_q_up(q: torch.Tensor, w: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor, *,
                    interleaved: bool = True, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The queries in the latent space (include/sparse_mla.h): per head the nope dims through w on the
    tensor cores, the rope dims rotated by the token's position; what sparse_mla_fwd takes as q.

    q [T, h, dn + 64] bf16 (dn = 128, 192 or 256 nope dims, then 64 rope dims), w [h, dn, 512] bf16,
    positions [T] int32 (-1 = unused token: zero rope dims), cos_sin [max_pos, 64] fp32 as in
    sparse_mla_append; returns out [T, h, 576] bf16.  Any other position out of range gives zero rope
    dims and makes the next sync_status() raise SMLA_ERR_INDEX_RANGE.
    """
    if q.dim() != 3 or q.dtype != _BF16 or not q.is_contiguous():
        raise ValueError("q must be a contiguous [T, h, dn + 64] bf16 tensor")
    T, h, d = q.shape
    dn = d - (D_QK - D_V)
    if w.shape != (h, dn, D_V) or w.dtype != _BF16 or not w.is_contiguous():
        raise ValueError(f"w must be a contiguous [{h}, {dn}, 512] bf16 tensor")
    max_pos = _positions_and_table(T, positions, cos_sin)
    dev = _cuda_device("q", q)
    if not dev == w.device == positions.device == cos_sin.device:
        _apart(dev, w=w, positions=positions, cos_sin=cos_sin)
    if out is None:
        out = _empty((T, h, D_QK), _BF16, dev, stream)
    else:
        if out.shape != (T, h, D_QK) or out.dtype != _BF16 or not out.is_contiguous():
            raise ValueError("out must be a contiguous [T, h, 576] bf16 tensor")
        if out.device != dev:
            _apart(dev, out=out)
    _call(dev, stream, library().sparse_mla_q_up, q.data_ptr(), w.data_ptr(), positions.data_ptr(), T, h, dn,
          cos_sin.data_ptr(), max_pos, 1 if interleaved else 0, out.data_ptr())
    return out


def _workspace(dev: torch.device, stream, workspace: Optional[torch.Tensor], bytes_of, *shape) -> Optional[torch.Tensor]:
    """The caller's workspace, or one for a call on `stream` of bytes_of(device, *shape) bytes (None: needs none)."""
    if workspace is not None:
        if workspace.dtype != _U8 or not workspace.is_contiguous() or workspace.device != dev:
            raise ValueError(f"workspace must be a contiguous uint8 tensor on {dev}")
        return workspace
    if torch.cuda.current_device() == dev.index:
        n = bytes_of(dev.index, *shape)
    else:
        with torch.cuda.device(dev):
            n = bytes_of(dev.index, *shape)
    return _empty((n,), _U8, dev, stream, result=False) if n else None


@functools.lru_cache(maxsize=1024)
def _prefix_workspace_bytes(device_index: int, T: int, h: int, prefix_len: int, fmt: int) -> int:
    """The library's answer for the device that is current, asked once per shape and device."""
    return int(library().sparse_mla_prefix_workspace_bytes(T, h, prefix_len, fmt))


def prefix_workspace_bytes(T: int, h: int, prefix_len: int, kv_format: str = "bf16") -> int:
    """Bytes of workspace that sparse_mla_prefix needs on the current device (0: none)."""
    if kv_format not in KV_FORMATS:
        raise ValueError(f"kv_format must be one of {sorted(KV_FORMATS)}")
    return int(library().sparse_mla_prefix_workspace_bytes(T, h, prefix_len, KV_FORMATS[kv_format]))


def sparse_mla_prefix(q: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor, prefix_len: int,
                      scale: Optional[float] = None, *, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None, kv_format: str = "bf16",
                      workspace: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of every token and head over one shared prefix (include/sparse_mla.h), its rows read
    once for the batch: q [T, h, 576] bf16, kv_cache as in sparse_mla_fwd, block_table
    [ceil(prefix_len / 64)] int32 (position i is slot block_table[i / 64] * 64 + i % 64).

    Returns out [T, h, 512] bf16 and lse [T, h] fp32, which sparse_mla_merge joins with each token's
    own part.  scale defaults to 576 ** -0.5.  workspace: a uint8 tensor of prefix_workspace_bytes(T,
    h, prefix_len, kv_format) bytes for callers that keep one (calls that may overlap need their own);
    allocated here otherwise, from torch's allocator on the stream of the call, as out and lse are.
    """
    if q.dim() != 3 or q.shape[2] != D_QK or q.dtype != _BF16 or not q.is_contiguous():
        raise ValueError(f"q must be a contiguous [T, h, 576] bf16 tensor, got {tuple(q.shape)} {q.dtype}")
    T, h, _ = q.shape
    prefix_len = int(prefix_len)
    num_slots = _cache_rows(kv_cache, kv_format)
    if prefix_len < 0 or block_table.dim() != 1 or block_table.dtype != _I32 \
            or block_table.numel() * 64 < prefix_len or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous [ceil(prefix_len / 64)] int32 tensor, prefix_len >= 0")
    dev = _cuda_device("q", q)
    if not dev == kv_cache.device == block_table.device:
        _apart(dev, kv_cache=kv_cache, block_table=block_table)
    if scale is None:
        scale = D_QK ** -0.5
    if out is None:
        out = _empty((T, h, D_V), _BF16, dev, stream)
    else:
        if out.shape != (T, h, D_V) or out.dtype != _BF16 or not out.is_contiguous():
            raise ValueError("out must be a contiguous [T, h, 512] bf16 tensor")
        if out.device != dev:
            _apart(dev, out=out)
    if lse is None:
        lse = _empty((T, h), _F32, dev, stream)
    else:
        if lse.shape != (T, h) or lse.dtype != _F32 or not lse.is_contiguous():
            raise ValueError("lse must be a contiguous [T, h] fp32 tensor")
        if lse.device != dev:
            _apart(dev, lse=lse)
    fmt = KV_FORMATS[kv_format]
    workspace = _workspace(dev, stream, workspace, _prefix_workspace_bytes, T, h, prefix_len, fmt)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    _call(dev, stream, library().sparse_mla_prefix, q.data_ptr(), kv_cache.data_ptr(), block_table.data_ptr(), T, h,
          prefix_len, num_slots, fmt, float(scale), out.data_ptr(), lse.data_ptr(), ws_ptr, ws_bytes)
    return out, lse


# ---- a batch of sequences, each over its own rows

@functools.lru_cache(maxsize=1024)
def _tree_workspace_bytes(device_index: int, T: int, h: int, seqs: int) -> int:
    """The library's answer for the device that is current, asked once per shape and device."""
    return int(library().sparse_mla_tree_workspace_bytes(T, h, seqs))


def tree_workspace_bytes(T: int, h: int, seqs: int) -> int:
    """Bytes of workspace that sparse_mla_tree needs on the current device."""
    return int(library().sparse_mla_tree_workspace_bytes(T, h, seqs))


def _batch(dev: torch.device, block_tables: torch.Tensor, lengths: torch.Tensor) -> Tuple[int, int]:
    """Sequences and blocks per sequence of a batch's tables."""
    shape = block_tables.shape
    if len(shape) != 2 or shape[1] < 1 or block_tables.dtype is not _I32 or not block_tables.is_contiguous():
        raise ValueError("block_tables must be a contiguous [seqs, blocks] int32 tensor of at least one block")
    seqs, blocks = shape
    if lengths.shape != (seqs,) or lengths.dtype is not _I32 or not lengths.is_contiguous():
        raise ValueError(f"lengths must be a contiguous [{seqs}] int32 tensor")
    if not dev == block_tables.device == lengths.device:
        _apart(dev, block_tables=block_tables, lengths=lengths)
    return seqs, blocks


def _tokens(dev: torch.device, T: int, seqs: int, starts: torch.Tensor, mask: Optional[torch.Tensor]):
    """Checks starts and the mask; the mask's pointer and words per token."""
    if starts.shape != (seqs + 1,) or starts.dtype is not _I32 or not starts.is_contiguous():
        raise ValueError(f"starts must be a contiguous [{seqs + 1}] int32 tensor")
    if starts.device != dev:
        _apart(dev, starts=starts)
    if mask is None:
        return None, 0
    shape = mask.shape
    if len(shape) != 2 or shape[0] != T or shape[1] < 1 or mask.dtype is not _I32 or not mask.is_contiguous():
        raise ValueError(f"mask must be a contiguous [{T}, words] int32 tensor of at least one word")
    if mask.device != dev:
        _apart(dev, mask=mask)
    return mask.data_ptr(), shape[1]


def _queries(q: torch.Tensor, kv_cache: torch.Tensor, kv_format: str) -> Tuple[torch.device, int, int, int]:
    """The device, tokens, heads and cache rows of a call on a batch."""
    shape = q.shape
    if len(shape) != 3 or shape[2] != D_QK or q.dtype is not _BF16 or not q.is_contiguous():
        raise ValueError(f"q must be a contiguous [T, h, 576] bf16 tensor, got {tuple(shape)} {q.dtype}")
    num_slots = _cache_rows(kv_cache, kv_format)
    dev = _cuda_device("q", q)
    if kv_cache.device != dev:
        _apart(dev, kv_cache=kv_cache)
    return dev, shape[0], shape[1], num_slots


def sparse_mla_tree(q: torch.Tensor, kv_cache: torch.Tensor, block_tables: torch.Tensor, lengths: torch.Tensor,
                    starts: torch.Tensor, scale: Optional[float] = None, *, mask: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, kv_format: str = "bf16",
                    workspace: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of each sequence's drafted tokens over its cached rows and the tree that they form
    (include/sparse_mla.h).

    q [T, h, 576] bf16, kv_cache as in sparse_mla_fwd, block_tables [seqs, blocks] int32, lengths [seqs]
    int32 (cached rows before the drafted ones), starts [seqs + 1] int32: sequence b's tokens are
    starts[b] .. starts[b + 1] - 1, the row of its j-th one at position lengths[b] + j.  mask [T, words]
    int32 bit words (as sparse_mla_scatter_mask writes them): bit j of a token's words lets it see
    drafted token j of its sequence; None: chains, each token sees those up to itself.

    Returns out [T, h, 512] bf16 and lse [T, h] fp32; tokens of no sequence are left as they are.
    scale defaults to 576 ** -0.5.  workspace: a uint8 tensor of tree_workspace_bytes(T, h, seqs) bytes
    for callers that keep one (calls that may overlap need their own); allocated here otherwise, from
    torch's allocator on the stream of the call, as out and lse are.
    """
    dev, T, h, num_slots = _queries(q, kv_cache, kv_format)
    seqs, blocks = _batch(dev, block_tables, lengths)
    mask_ptr, words = _tokens(dev, T, seqs, starts, mask)
    if scale is None:
        scale = D_QK ** -0.5
    out = _empty((T, h, D_V), _BF16, dev, stream) if out is None else _given("out", out, (T, h, D_V), _BF16, dev)
    lse = _empty((T, h), _F32, dev, stream) if lse is None else _given("lse", lse, (T, h), _F32, dev)
    workspace = _workspace(dev, stream, workspace, _tree_workspace_bytes, T, h, seqs)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    _call(dev, stream, library().sparse_mla_tree, q.data_ptr(), kv_cache.data_ptr(), block_tables.data_ptr(),
          lengths.data_ptr(), starts.data_ptr(), mask_ptr, T, h, seqs, blocks, words, num_slots, KV_FORMATS[kv_format],
          float(scale), out.data_ptr(), lse.data_ptr(), ws_ptr, ws_bytes)
    return out, lse


def sparse_mla_weights(q: torch.Tensor, kv_cache: torch.Tensor, block_tables: torch.Tensor, lengths: torch.Tensor,
                       starts: torch.Tensor, lse: torch.Tensor, scale: Optional[float] = None, *,
                       mask: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None, decay: float = 1.0,
                       out: Optional[torch.Tensor] = None, kv_format: str = "bf16", stream=None) -> torch.Tensor:
    """The attention weight that every cached row has gathered (include/sparse_mla.h): per sequence and
    position decay * weights, plus the probabilities of its tokens and heads there.

    q, kv_cache, block_tables, lengths, starts, scale and mask as in sparse_mla_tree, lse [T, h] fp32 as
    it returned it.  weights [seqs, blocks * 64] fp32 are what earlier calls gathered (None: nothing yet);
    returns out of the same shape, which may be passed in and may be weights itself.
    Of drafted tokens, gather from the accepted ones, as a chain, when their rows have been appended behind
    the cached ones.
    """
    dev, T, h, num_slots = _queries(q, kv_cache, kv_format)
    seqs, blocks = _batch(dev, block_tables, lengths)
    mask_ptr, words = _tokens(dev, T, seqs, starts, mask)
    _given("lse", lse, (T, h), _F32, dev)
    prev = None if weights is None else _given("weights", weights, (seqs, blocks * 64), _F32, dev).data_ptr()
    if scale is None:
        scale = D_QK ** -0.5
    out = (_empty((seqs, blocks * 64), _F32, dev, stream) if out is None
           else _given("out", out, (seqs, blocks * 64), _F32, dev))
    _call(dev, stream, library().sparse_mla_weights, q.data_ptr(), kv_cache.data_ptr(), block_tables.data_ptr(),
          lengths.data_ptr(), starts.data_ptr(), mask_ptr, lse.data_ptr(), prev, float(decay), T, h, seqs, blocks, words,
          num_slots, KV_FORMATS[kv_format], float(scale), out.data_ptr())
    return out


def sparse_mla_evict(kv_cache: torch.Tensor, block_tables: torch.Tensor, lengths: torch.Tensor, weights: torch.Tensor,
                     new_tables: torch.Tensor, budget: int, *, sinks: int = 0, recent: int = 0, kv_format: str = "bf16",
                     kept: Optional[torch.Tensor] = None, new_lengths: Optional[torch.Tensor] = None,
                     new_weights: Optional[torch.Tensor] = None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Shrink each sequence's cache to `budget` rows by gathered attention weight (include/sparse_mla.h):
    the first `sinks` rows, the last `recent` ones and the heaviest between them, ties to the lower
    position, copied in order into the pages of new_tables.

    block_tables [seqs, blocks] int32, lengths [seqs] int32, weights [seqs, blocks * 64] fp32 as
    sparse_mla_weights gives them, new_tables [seqs, new_blocks] int32: pages of the same cache that
    hold no row of any sequence.  Returns kept [seqs, budget] int32 (positions, ascending, then -1),
    new_lengths [seqs] int32 and new_weights [seqs, new_blocks * 64] fp32; passed in, they are tensors of
    their own (new_lengths is not lengths, nor new_weights weights: refused).  A row that lies or would go
    outside the cache is not copied and makes the next sync_status() raise SMLA_ERR_INDEX_RANGE.
    """
    num_slots = _cache_rows(kv_cache, kv_format)
    dev = _cuda_device("kv_cache", kv_cache)
    seqs, blocks = _batch(dev, block_tables, lengths)
    if weights.shape != (seqs, blocks * 64) or weights.dtype != _F32 or not weights.is_contiguous():
        raise ValueError(f"weights must be a contiguous [{seqs}, {blocks * 64}] fp32 tensor")
    if new_tables.dim() != 2 or new_tables.shape[0] != seqs or new_tables.dtype != _I32 or not new_tables.is_contiguous():
        raise ValueError(f"new_tables must be a contiguous [{seqs}, new_blocks] int32 tensor")
    if not dev == weights.device == new_tables.device:
        _apart(dev, weights=weights, new_tables=new_tables)
    new_blocks = new_tables.shape[1]
    budget, sinks, recent = int(budget), int(sinks), int(recent)
    if not 1 <= budget <= new_blocks * 64:
        raise ValueError(f"budget must be in [1, {new_blocks * 64}], the positions of new_tables")
    if sinks < 0 or recent < 0 or sinks + recent > budget:
        raise ValueError("sinks and recent must be >= 0 and no more than the budget together")
    kept = _empty((seqs, budget), _I32, dev, stream) if kept is None else _given("kept", kept, (seqs, budget), _I32, dev)
    new_lengths = _empty((seqs,), _I32, dev, stream) if new_lengths is None else _given("new_lengths", new_lengths, (seqs,), _I32, dev)
    width = new_blocks * 64
    new_weights = (_empty((seqs, width), _F32, dev, stream) if new_weights is None
                   else _given("new_weights", new_weights, (seqs, width), _F32, dev))
    _call(dev, stream, library().sparse_mla_evict, kv_cache.data_ptr(), block_tables.data_ptr(), lengths.data_ptr(),
          weights.data_ptr(), new_tables.data_ptr(), seqs, blocks, new_blocks, budget, sinks, recent, num_slots,
          KV_FORMATS[kv_format], kept.data_ptr(), new_lengths.data_ptr(), new_weights.data_ptr())
    return kept, new_lengths, new_weights


def host_workspace_bytes(T: int, h: int, topk: int) -> int:
    return int(library().sparse_mla_host_workspace_bytes(T, h, topk))


def sparse_mla_fwd_host(q_host: torch.Tensor, kv_cache: torch.Tensor, indices_host: torch.Tensor,
                        scale: float, out_host: torch.Tensor, lse_host: torch.Tensor,
                        workspace: torch.Tensor, *, kv_format: str = "bf16", stream=None) -> None:
    """Forward pass with host-resident q/indices/out/lse (pinned for async copies);
    the library queues H2D copies, the kernel and D2H copies on `stream`."""
    T, h, topk, num_slots = _dims(q_host, kv_cache, indices_host, kv_format)
    if q_host.is_cuda or indices_host.is_cuda or out_host.is_cuda or lse_host.is_cuda:
        raise ValueError("q, indices, out and lse must be host tensors here")
    dev = _device_of((("kv_cache", kv_cache), ("workspace", workspace)))
    with _on(dev):
        st = library().sparse_mla_fwd_host(
            q_host.data_ptr(), kv_cache.data_ptr(), indices_host.data_ptr(), T, h, topk,
            num_slots, KV_FORMATS[kv_format], float(scale), out_host.data_ptr(),
            lse_host.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
            _stream_handle(stream, dev))
    _check(st)


@functools.lru_cache(maxsize=256)
def _host_io_layout(T: int, h: int, topk: int) -> Tuple[int, int, int, int]:
    a, b, c, d = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(library().sparse_mla_host_io_layout(T, h, topk, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c),
                                               ctypes.byref(d)))
    return a.value, b.value, c.value, d.value


def host_io_layout(T: int, h: int, topk: int) -> dict:
    """Sizes and offsets of the packed host buffers of sparse_mla_fwd_host_packed (the library's
    answer, asked once per shape)."""
    a, b, c, d = _host_io_layout(int(T), int(h), int(topk))
    return {"in_bytes": a, "indices_offset": b, "out_bytes": c, "lse_offset": d}


def host_io_views(in_host: torch.Tensor, out_host: torch.Tensor, T: int, h: int, topk: int):
    """Views of q / indices inside a packed input buffer and of out / lse inside a packed output
    buffer (uint8 host tensors of the sizes host_io_layout gives)."""
    lay = host_io_layout(T, h, topk)
    if in_host.dtype != torch.uint8 or in_host.numel() < lay["in_bytes"]:
        raise ValueError(f"in_host must be a uint8 tensor of at least {lay['in_bytes']} bytes")
    if out_host.dtype != torch.uint8 or out_host.numel() < lay["out_bytes"]:
        raise ValueError(f"out_host must be a uint8 tensor of at least {lay['out_bytes']} bytes")
    i0, l0 = lay["indices_offset"], lay["lse_offset"]
    q = in_host[: T * h * D_QK * 2].view(torch.bfloat16).view(T, h, D_QK)
    idx = in_host[i0: i0 + T * topk * 4].view(torch.int32).view(T, topk)
    out = out_host[: T * h * D_V * 2].view(torch.bfloat16).view(T, h, D_V)
    lse = out_host[l0: l0 + T * h * 4].view(torch.float32).view(T, h)
    return q, idx, out, lse


def sparse_mla_fwd_host_packed(in_host: torch.Tensor, kv_cache: torch.Tensor, T: int, h: int, topk: int,
                               scale: float, out_host: torch.Tensor, workspace: torch.Tensor, *,
                               kv_format: str = "bf16", stream=None) -> None:
    """Forward pass from one packed host input buffer into one packed host output buffer
    (include/sparse_mla.h): one H2D copy, the kernel and one D2H copy queued on `stream`."""
    if in_host.is_cuda or out_host.is_cuda:
        raise ValueError("in_host and out_host must be host tensors")
    for name, t in (("in_host", in_host), ("out_host", out_host)):
        if t.dtype != torch.uint8 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous uint8 tensor")
    if kv_format not in KV_FORMATS:
        raise ValueError(f"kv_format must be one of {sorted(KV_FORMATS)}")
    in_bytes, _, out_bytes, _ = _host_io_layout(int(T), int(h), int(topk))
    if in_host.numel() < in_bytes or out_host.numel() < out_bytes:
        raise ValueError("in_host / out_host smaller than host_io_layout says")
    dev = _device_of((("kv_cache", kv_cache), ("workspace", workspace)))
    with _on(dev):
        st = library().sparse_mla_fwd_host_packed(
            in_host.data_ptr(), kv_cache.data_ptr(), T, h, topk, int(kv_cache.shape[0]),
            KV_FORMATS[kv_format], float(scale), out_host.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _stream_handle(stream, dev))
    _check(st)


def sync_status(stream=None) -> None:
    """Synchronise the stream and raise if a kernel reported a device-side error."""
    _check(library().sparse_mla_sync_status(_stream_handle(stream)))


def launch_info(T: int, h: int, topk: int, kv_format: str = "bf16") -> dict:
    s, c, m, n = (ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32())
    _check(library().sparse_mla_launch_info(T, h, topk, KV_FORMATS[kv_format], ctypes.byref(s),
                                            ctypes.byref(c), ctypes.byref(m), ctypes.byref(n)))
    return {"splits": s.value, "ctas": c.value, "smem_bytes": m.value, "launches": n.value}
