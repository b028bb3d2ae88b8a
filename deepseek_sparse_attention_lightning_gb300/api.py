"""ctypes binding of libdsa.so: the C ABI of include/dsa.h, same names.

Argument marshalling only: every step of the decode path runs in the
library's CUDA kernels.  Tensors are torch CUDA tensors (torch provides device
memory and streams); each wrapper checks dtype, device and contiguity, passes
raw pointers, and raises ``DSAError`` on a non-zero status.  There is no CPU
fallback: without the built library every call raises.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import c_float, c_int32, c_int64, c_size_t, c_void_p

import torch

from . import build as _build

DSA_OK = 0
STATUS_NAMES = {0: "DSA_OK", 1: "DSA_ERR_INVALID_ARG", 2: "DSA_ERR_UNSUPPORTED",
                3: "DSA_ERR_WORKSPACE", 4: "DSA_ERR_CUDA", 5: "DSA_ERR_DEVICE_CHECK",
                6: "DSA_ERR_TIMEOUT"}
PAGE_SIZE = 64


class DSAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


class DecodeDesc(ctypes.Structure):
    _fields_ = [("batch", c_int32), ("q_per_req", c_int32), ("num_heads", c_int32),
                ("topk", c_int32), ("page_size", c_int32), ("max_pages", c_int32),
                ("num_pages", c_int32), ("seqlens", c_void_p), ("page_table", c_void_p)]


class StepRing(ctypes.Structure):
    """The caller-owned resources of a ring of decode steps (dsa_step_ring)."""
    _fields_ = [("dev_in", c_void_p * 2), ("out", c_void_p * 2), ("ws", c_void_p),
                ("ws_bytes", c_size_t), ("copy_in_stream", c_void_p), ("copy_out_stream", c_void_p),
                ("ev_in", c_void_p * 2), ("ev_done", c_void_p * 2), ("ev_out", c_void_p * 2),
                ("step", c_int64)]


class StepLayout(ctypes.Structure):
    """Byte offsets of a decode step's inputs in one host/device block."""
    _fields_ = [("q_fp8", c_size_t), ("q_scale", c_size_t), ("w", c_size_t), ("q", c_size_t),
                ("seqlens", c_size_t), ("page_table", c_size_t), ("bytes", c_size_t)]


_SIGS = {
    "dsa_indexer_logits": (c_int32, [ctypes.POINTER(DecodeDesc), c_void_p, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_void_p, c_int64, c_void_p]),
    "dsa_topk": (c_int32, [ctypes.POINTER(DecodeDesc), c_void_p, c_int64, c_void_p, c_void_p,
                           c_size_t, c_void_p]),
    "dsa_topk_workspace_bytes": (c_size_t, [ctypes.POINTER(DecodeDesc), c_int64]),
    "dsa_topk_noalloc": (c_int32, [ctypes.POINTER(DecodeDesc), c_void_p, c_int64, c_void_p,
                                   c_void_p]),
    "dsa_sparse_mla_decode_split": (c_int32, [ctypes.POINTER(DecodeDesc), c_void_p, c_void_p,
                                              c_void_p, c_int32, c_float, c_void_p, c_void_p,
                                              c_void_p]),
    "dsa_merge": (c_int32, [c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "dsa_cache_write": (c_int32, [ctypes.POINTER(DecodeDesc), c_void_p, c_void_p, c_void_p,
                                  c_void_p, c_void_p, c_void_p]),
    "dsa_decode_fused": (c_int32, [ctypes.POINTER(DecodeDesc), c_void_p, c_void_p, c_void_p,
                                   c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                   c_float, c_int32, c_int32, c_void_p, c_void_p, c_size_t,
                                   c_void_p]),
    "dsa_decode_fused_timed": (c_int32, [ctypes.POINTER(DecodeDesc), c_void_p, c_void_p, c_void_p,
                                         c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                         c_void_p, c_float, c_int32, c_int32, c_void_p, c_void_p,
                                         c_size_t, c_void_p, ctypes.POINTER(c_void_p)]),
    "dsa_decode_fused_write": (c_int32, [ctypes.POINTER(DecodeDesc), c_void_p, c_void_p, c_void_p,
                                         c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                         c_void_p, c_void_p, c_void_p, c_float, c_int32, c_int32,
                                         c_void_p, c_void_p, c_size_t, c_void_p]),
    "dsa_latent_to_fp8": (c_int32, [c_void_p, c_int64, c_void_p, c_void_p]),
    "dsa_sparse_mla_decode_split_fp8": (c_int32, [ctypes.POINTER(DecodeDesc), c_void_p, c_void_p,
                                                  c_void_p, c_int32, c_float, c_void_p, c_void_p,
                                                  c_void_p]),
    "dsa_decode_fused_fp8kv": (c_int32, [ctypes.POINTER(DecodeDesc), c_void_p, c_void_p, c_void_p,
                                         c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                         c_void_p, c_float, c_int32, c_int32, c_void_p, c_void_p,
                                         c_size_t, c_void_p]),
    "dsa_mla_decode": (c_int32, [ctypes.POINTER(DecodeDesc), c_void_p, c_void_p, c_float, c_void_p,
                                 c_void_p, c_void_p, c_size_t, c_void_p]),
    "dsa_mla_decode_fp8kv": (c_int32, [ctypes.POINTER(DecodeDesc), c_void_p, c_void_p, c_float,
                                       c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "dsa_mla_decode_workspace_bytes": (c_size_t, [ctypes.POINTER(DecodeDesc)]),
    "dsa_mla_prefill": (c_int32, [c_int32, c_int32, c_int32, c_int32, c_int32, c_void_p, c_void_p,
                                  c_void_p, c_void_p, c_void_p, c_int64, c_float, c_int32, c_void_p,
                                  c_void_p, c_void_p]),
    "dsa_pages_update": (c_int32, [c_int32, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                   c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p,
                                   c_void_p]),
    "dsa_kv_write": (c_int32, [c_int32, c_int32, c_int32, c_void_p, c_int64, c_void_p, c_int64,
                               c_void_p, c_int32, c_void_p, c_void_p, c_void_p]),
    "dsa_kv_write_fp8": (c_int32, [c_int32, c_int32, c_int32, c_void_p, c_int64, c_void_p, c_int64,
                                   c_void_p, c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                   c_void_p]),
    "dsa_gqa_decode": (c_int32, [ctypes.POINTER(DecodeDesc), c_int32, c_int32, c_void_p, c_void_p,
                                 c_void_p, c_float, c_void_p, c_void_p, c_void_p, c_size_t,
                                 c_void_p]),
    "dsa_gqa_decode_fp8kv": (c_int32, [ctypes.POINTER(DecodeDesc), c_int32, c_int32, c_void_p,
                                       c_void_p, c_void_p, c_void_p, c_void_p, c_float, c_void_p,
                                       c_void_p, c_void_p, c_size_t, c_void_p]),
    "dsa_gqa_decode_workspace_bytes": (c_size_t, [ctypes.POINTER(DecodeDesc), c_int32, c_int32]),
    "dsa_gqa_prefill": (c_int32, [c_int32, c_int32, c_int32, c_int32, c_int32, c_int32, c_int32,
                                  c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_int64, c_void_p,
                                  c_int64, c_float, c_int32, c_void_p, c_void_p, c_void_p]),
    "dsa_rmsnorm": (c_int32, [c_int32, c_int32, c_void_p, c_int64, c_void_p, c_void_p, c_float,
                              c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "dsa_decode_mli": (c_int32, [ctypes.POINTER(DecodeDesc), c_void_p, c_void_p, c_void_p,
                                 c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                 c_float, c_int32, c_int32, c_void_p, c_void_p, c_size_t,
                                 c_void_p]),
    "dsa_num_splits_mli": (c_int32, [ctypes.POINTER(DecodeDesc)]),
    "dsa_step_layout_get": (c_int32, [c_int32, c_int32, c_int32, c_int32,
                                      ctypes.POINTER(StepLayout)]),
    "dsa_decode_step_host": (c_int32, [ctypes.POINTER(DecodeDesc), c_void_p, c_void_p, c_void_p,
                                       c_void_p, c_void_p, c_float, c_int32, c_int32, c_void_p,
                                       c_void_p, c_void_p, c_size_t, c_void_p]),
    "dsa_decode_step_ring": (c_int32, [ctypes.POINTER(DecodeDesc), ctypes.POINTER(StepRing),
                                       c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_float,
                                       c_int32, c_int32, c_void_p]),
    "dsa_workspace_bytes": (c_size_t, [ctypes.POINTER(DecodeDesc), c_int32, c_int32]),
    "dsa_num_splits_auto": (c_int32, [ctypes.POINTER(DecodeDesc)]),
    "dsa_status_str": (ctypes.c_char_p, [c_int32]),
    "dsa_get_device_error": (c_int32, [c_void_p]),
    "dsa_version": (ctypes.c_char_p, []),
    "dsa_debug_set_wait_cycles": (c_int32, [c_int64]),
}

_lib = None


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """Loads libdsa.so (built in-tree by ``build.build()``); raises if absent."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libdsa.so not built at {path}: run "
                               "`python -c 'import __graft_entry__ as g; g.build()'` first")
        L = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != DSA_OK:
        raise DSAError(status, where)


def _ptr(t, dtype, name, ndim=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dims, got {t.dim()}")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _u16(t: torch.Tensor, name):
    if t.dtype == torch.bfloat16:
        return _ptr(t, torch.bfloat16, name)
    return _ptr(t, torch.int16, name)


def make_desc(seqlens: torch.Tensor, page_table: torch.Tensor, q_per_req: int, num_heads: int,
              topk: int, num_pages: int) -> DecodeDesc:
    """Descriptor of one decode batch (keeps no reference to the tensors)."""
    B = int(seqlens.shape[0])
    return DecodeDesc(batch=B, q_per_req=int(q_per_req), num_heads=int(num_heads),
                      topk=int(topk), page_size=PAGE_SIZE, max_pages=int(page_table.shape[1]),
                      num_pages=int(num_pages),
                      seqlens=_ptr(seqlens, torch.int32, "seqlens", 1),
                      page_table=_ptr(page_table, torch.int32, "page_table", 2))


def dsa_indexer_logits(desc, q_fp8, q_scale, w, k_fp8, k_scale, logits, ld=None, stream=None):
    ld = int(logits.shape[-1]) if ld is None else int(ld)
    _check(lib().dsa_indexer_logits(
        ctypes.byref(desc), _ptr(q_fp8, torch.uint8, "q_fp8"), _ptr(q_scale, torch.float32, "q_scale"),
        _ptr(w, torch.float32, "w"), _ptr(k_fp8, torch.uint8, "k_fp8"),
        _ptr(k_scale, torch.float32, "k_scale"), _ptr(logits, torch.float32, "logits"), ld,
        _stream(stream)), "dsa_indexer_logits")


def dsa_topk_workspace_bytes(desc, ld) -> int:
    return int(lib().dsa_topk_workspace_bytes(ctypes.byref(desc), int(ld)))


def dsa_topk(desc, logits, topk_idx, ws, ld=None, stream=None):
    ld = int(logits.shape[-1]) if ld is None else int(ld)
    _check(lib().dsa_topk(ctypes.byref(desc), _ptr(logits, torch.float32, "logits"), ld,
                          _ptr(topk_idx, torch.int32, "topk_idx"), _ptr(ws, torch.uint8, "ws"),
                          ws.numel(), _stream(stream)), "dsa_topk")


def dsa_topk_noalloc(desc, logits, topk_idx, ld=None, stream=None):
    """dsa_topk with the library's fixed device scratch instead of a workspace
    (for callers that cannot allocate device memory; see include/dsa.h)."""
    ld = int(logits.shape[-1]) if ld is None else int(ld)
    _check(lib().dsa_topk_noalloc(ctypes.byref(desc), _ptr(logits, torch.float32, "logits"), ld,
                                  _ptr(topk_idx, torch.int32, "topk_idx"), _stream(stream)),
           "dsa_topk_noalloc")


def dsa_sparse_mla_decode_split(desc, q, kv, topk_idx, num_splits, sm_scale, mid_o, mid_lse,
                                stream=None):
    _check(lib().dsa_sparse_mla_decode_split(
        ctypes.byref(desc), _u16(q, "q"), _u16(kv, "kv"), _ptr(topk_idx, torch.int32, "topk_idx"),
        int(num_splits), float(sm_scale), _ptr(mid_o, torch.float32, "mid_o"),
        _ptr(mid_lse, torch.float32, "mid_lse"), _stream(stream)), "dsa_sparse_mla_decode_split")


def dsa_cache_write(desc, new_latent, new_index_k, kv, k_fp8, k_scale, stream=None):
    _check(lib().dsa_cache_write(ctypes.byref(desc), _ptr(new_latent, torch.bfloat16, "new_latent"),
                                 _ptr(new_index_k, torch.bfloat16, "new_index_k"),
                                 _ptr(kv, torch.bfloat16, "kv"), _ptr(k_fp8, torch.uint8, "k_fp8"),
                                 _ptr(k_scale, torch.float32, "k_scale"), _stream(stream)),
           "dsa_cache_write")


def dsa_merge(num_rows, num_splits, mid_o, mid_lse, out, out_lse=None, stream=None):
    _check(lib().dsa_merge(int(num_rows), int(num_splits), _ptr(mid_o, torch.float32, "mid_o"),
                           _ptr(mid_lse, torch.float32, "mid_lse"), _ptr(out, torch.float32, "out"),
                           _ptr(out_lse, torch.float32, "out_lse"), _stream(stream)), "dsa_merge")


def dsa_workspace_bytes(desc, max_seqlen, num_splits=0) -> int:
    return int(lib().dsa_workspace_bytes(ctypes.byref(desc), int(max_seqlen), int(num_splits)))


def dsa_num_splits_auto(desc) -> int:
    return int(lib().dsa_num_splits_auto(ctypes.byref(desc)))


def dsa_decode_fused(desc, q_fp8, q_scale, w, k_fp8, k_scale, q, kv, out, ws, max_seqlen,
                     sm_scale, num_splits=0, topk_in=None, topk_out=None, stream=None,
                     stage_events=None):
    """``stage_events``: optional list of 5 torch.cuda.Event (timing enabled)."""
    if stage_events is not None:
        arr = (c_void_p * 5)(*[ev.cuda_event if ev is not None else None for ev in stage_events])
        _check(lib().dsa_decode_fused_timed(
            ctypes.byref(desc), _ptr(q_fp8, torch.uint8, "q_fp8"),
            _ptr(q_scale, torch.float32, "q_scale"), _ptr(w, torch.float32, "w"),
            _ptr(k_fp8, torch.uint8, "k_fp8"), _ptr(k_scale, torch.float32, "k_scale"),
            _u16(q, "q"), _u16(kv, "kv"), _ptr(topk_in, torch.int32, "topk_in"),
            _ptr(topk_out, torch.int32, "topk_out"), float(sm_scale), int(num_splits),
            int(max_seqlen), _ptr(out, torch.float32, "out"), _ptr(ws, torch.uint8, "ws"),
            ws.numel(), _stream(stream), arr), "dsa_decode_fused_timed")
        return
    _check(lib().dsa_decode_fused(
        ctypes.byref(desc), _ptr(q_fp8, torch.uint8, "q_fp8"), _ptr(q_scale, torch.float32, "q_scale"),
        _ptr(w, torch.float32, "w"), _ptr(k_fp8, torch.uint8, "k_fp8"),
        _ptr(k_scale, torch.float32, "k_scale"), _u16(q, "q"), _u16(kv, "kv"),
        _ptr(topk_in, torch.int32, "topk_in"), _ptr(topk_out, torch.int32, "topk_out"),
        float(sm_scale), int(num_splits), int(max_seqlen), _ptr(out, torch.float32, "out"),
        _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)), "dsa_decode_fused")


def dsa_decode_fused_write(desc, new_latent, new_index_k, q_fp8, q_scale, w, k_fp8, k_scale, q,
                           kv, out, ws, max_seqlen, sm_scale, num_splits=0, topk_in=None,
                           topk_out=None, stream=None):
    _check(lib().dsa_decode_fused_write(
        ctypes.byref(desc), _ptr(new_latent, torch.bfloat16, "new_latent"),
        _ptr(new_index_k, torch.bfloat16, "new_index_k"), _ptr(q_fp8, torch.uint8, "q_fp8"),
        _ptr(q_scale, torch.float32, "q_scale"), _ptr(w, torch.float32, "w"),
        _ptr(k_fp8, torch.uint8, "k_fp8"), _ptr(k_scale, torch.float32, "k_scale"), _u16(q, "q"),
        _u16(kv, "kv"), _ptr(topk_in, torch.int32, "topk_in"),
        _ptr(topk_out, torch.int32, "topk_out"), float(sm_scale), int(num_splits),
        int(max_seqlen), _ptr(out, torch.float32, "out"), _ptr(ws, torch.uint8, "ws"),
        ws.numel(), _stream(stream)), "dsa_decode_fused_write")


def dsa_latent_to_fp8(kv, kv8, stream=None):
    rows = int(kv.shape[0])
    if kv8.shape != (rows, 656):
        raise ValueError("kv8 must be [rows, 656]")
    _check(lib().dsa_latent_to_fp8(_u16(kv, "kv"), rows, _ptr(kv8, torch.uint8, "kv8"),
                                   _stream(stream)), "dsa_latent_to_fp8")


def dsa_sparse_mla_decode_split_fp8(desc, q, kv8, topk_idx, num_splits, sm_scale, mid_o, mid_lse,
                                    stream=None):
    _check(lib().dsa_sparse_mla_decode_split_fp8(
        ctypes.byref(desc), _u16(q, "q"), _ptr(kv8, torch.uint8, "kv8"),
        _ptr(topk_idx, torch.int32, "topk_idx"), int(num_splits), float(sm_scale),
        _ptr(mid_o, torch.float32, "mid_o"), _ptr(mid_lse, torch.float32, "mid_lse"),
        _stream(stream)), "dsa_sparse_mla_decode_split_fp8")


def dsa_decode_fused_fp8kv(desc, q_fp8, q_scale, w, k_fp8, k_scale, q, kv8, out, ws, max_seqlen,
                           sm_scale, num_splits=0, topk_in=None, topk_out=None, stream=None):
    _check(lib().dsa_decode_fused_fp8kv(
        ctypes.byref(desc), _ptr(q_fp8, torch.uint8, "q_fp8"), _ptr(q_scale, torch.float32, "q_scale"),
        _ptr(w, torch.float32, "w"), _ptr(k_fp8, torch.uint8, "k_fp8"),
        _ptr(k_scale, torch.float32, "k_scale"), _u16(q, "q"), _ptr(kv8, torch.uint8, "kv8"),
        _ptr(topk_in, torch.int32, "topk_in"), _ptr(topk_out, torch.int32, "topk_out"),
        float(sm_scale), int(num_splits), int(max_seqlen), _ptr(out, torch.float32, "out"),
        _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)), "dsa_decode_fused_fp8kv")


def _arg(t, dtype, shape, dev, name):
    """Pointer of a contiguous tensor of that dtype and shape on CUDA device ``dev`` (None: NULL).  One
    combined test for the usual case: a small launch is bound by what the host does before it."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor")
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on the current device cuda:{dev}, got {t.device}")
    raise ValueError(f"{name}: expected a contiguous tensor")


def _rows_arg(t, dtype, dev, name):
    """(pointer, row stride) of a 2-D tensor with contiguous columns; its rows may be strided."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.dim() != 2:
        raise TypeError(f"{name}: expected a 2-D {dtype} tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on the current device cuda:{dev}, got {t.device}")
    rows, cols = t.shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name}: expected contiguous columns")
    return t.data_ptr(), (ld if rows > 1 else cols)


def _heads_arg(t, shape, dev, name):
    """(pointer, row stride) of a bf16 tensor [rows, heads, dim] whose heads lie side by side; its rows may
    be strided (columns of a wider projection)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.dim() != 3:
        raise TypeError(f"{name}: expected a 3-D {torch.bfloat16} tensor")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on the current device cuda:{dev}, got {t.device}")
    rows, heads, dim = shape
    ld, hs, step = t.stride()
    if (dim > 1 and step != 1) or (heads > 1 and hs != dim):
        raise ValueError(f"{name}: expected contiguous heads")
    return t.data_ptr(), (ld if rows > 1 else heads * dim)


def _stream_on(stream, dev) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return _stream(stream)


def dsa_mla_decode_workspace_bytes(desc) -> int:
    return int(lib().dsa_mla_decode_workspace_bytes(ctypes.byref(desc)))


def dsa_mla_decode(desc, q, kv, out, ws, sm_scale, lse=None, stream=None):
    """Dense latent attention over the paged cache (every visible token): ``out`` bf16 [T, H, 512],
    ``lse`` float32 [T, H] or None; see include/dsa.h."""
    fn, dev, bf16 = lib().dsa_mla_decode, torch.cuda.current_device(), torch.bfloat16
    T, H = desc.batch * desc.q_per_req, desc.num_heads
    _check(fn(ctypes.byref(desc), _arg(q, bf16, (T, H, 576), dev, "q"),
              _arg(kv, bf16, (desc.num_pages * PAGE_SIZE, 576), dev, "kv"), sm_scale,
              _arg(out, bf16, (T, H, 512), dev, "out"), _arg(lse, torch.float32, (T, H), dev, "lse"),
              _arg(ws, torch.uint8, (ws.numel(),), dev, "ws"), ws.numel(), _stream_on(stream, dev)),
           "dsa_mla_decode")


def dsa_mla_decode_fp8kv(desc, q, kv8, out, ws, sm_scale, lse=None, stream=None):
    """dsa_mla_decode over the FP8 latent cache ``kv8`` (uint8 [num_pages * 64, 656])."""
    fn, dev, bf16 = lib().dsa_mla_decode_fp8kv, torch.cuda.current_device(), torch.bfloat16
    T, H = desc.batch * desc.q_per_req, desc.num_heads
    _check(fn(ctypes.byref(desc), _arg(q, bf16, (T, H, 576), dev, "q"),
              _arg(kv8, torch.uint8, (desc.num_pages * PAGE_SIZE, 656), dev, "kv8"), sm_scale,
              _arg(out, bf16, (T, H, 512), dev, "out"), _arg(lse, torch.float32, (T, H), dev, "lse"),
              _arg(ws, torch.uint8, (ws.numel(),), dev, "ws"), ws.numel(), _stream_on(stream, dev)),
           "dsa_mla_decode_fp8kv")


def dsa_mla_prefill(q, kv, k_rope, cu_q, cu_k, out, max_q, sm_scale, causal=True, lse=None,
                    stream=None):
    """Attention of packed prompts over expanded keys and values: ``q`` [total_q, H, 192], ``kv``
    [total_k, H, 256] (key 128, value 128), ``k_rope`` [total_k, 64] (rows may be strided: the last 64
    columns of latent rows), ``out`` [total_q, H, 128], all bf16; see include/dsa.h."""
    fn, dev, bf16, i32 = lib().dsa_mla_prefill, torch.cuda.current_device(), torch.bfloat16, torch.int32
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise TypeError("q: expected a 3-D tensor")
    if not isinstance(cu_q, torch.Tensor) or cu_q.dim() != 1 or cu_q.shape[0] < 2:
        raise TypeError("cu_q: expected a 1-D tensor of at least two offsets")
    rp, ld = _rows_arg(k_rope, bf16, dev, "k_rope")
    Tq, H, _ = q.shape
    Tk, B1 = k_rope.shape[0], cu_q.shape[0]
    if k_rope.shape[1] != 64:
        raise ValueError(f"k_rope: expected 64 columns, got {k_rope.shape[1]}")
    _check(fn(B1 - 1, H, Tq, Tk, max_q, _arg(cu_q, i32, (B1,), dev, "cu_q"),
              _arg(cu_k, i32, (B1,), dev, "cu_k"), _arg(q, bf16, (Tq, H, 192), dev, "q"),
              _arg(kv, bf16, (Tk, H, 256), dev, "kv"), rp, ld, sm_scale, 1 if causal else 0,
              _arg(out, bf16, (Tq, H, 128), dev, "out"),
              _arg(lse, torch.float32, (Tq, H), dev, "lse"), _stream_on(stream, dev)),
           "dsa_mla_prefill")


def dsa_pages_update(change, seqlens, page_table, free_pages, free_count, cu_new, slots, seqlens_out=None,
                     free_count_out=None, stream=None):
    """Pages and cache rows for the ``change`` [B] new tokens of each request (negative: it has ended and
    gives its pages back), from the stack ``free_pages`` [num_pages] of ``free_count`` [1] pages: updates
    ``page_table`` [B, max_pages], ``seqlens`` and ``free_count`` (or writes the new ones to ``seqlens_out``
    and ``free_count_out``), writes ``cu_new`` [B + 1] and ``slots`` [max_tokens]; all int32; see
    include/dsa.h."""
    fn, dev, i32 = lib().dsa_pages_update, torch.cuda.current_device(), torch.int32
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise TypeError("page_table: expected a 2-D tensor")
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise TypeError("free_pages: expected a 1-D tensor")
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise TypeError("slots: expected a 1-D tensor")
    B, max_pages = page_table.shape
    num_pages, max_tokens = free_pages.shape[0], slots.shape[0]
    seq, cnt = _arg(seqlens, i32, (B,), dev, "seqlens"), _arg(free_count, i32, (1,), dev, "free_count")
    _check(fn(B, max_pages, num_pages, _arg(change, i32, (B,), dev, "change"), seq,
              seq if seqlens_out is None else _arg(seqlens_out, i32, (B,), dev, "seqlens_out"),
              _arg(page_table, i32, (B, max_pages), dev, "page_table"),
              _arg(free_pages, i32, (num_pages,), dev, "free_pages"), cnt,
              cnt if free_count_out is None else _arg(free_count_out, i32, (1,), dev, "free_count_out"),
              max_tokens, _arg(cu_new, i32, (B + 1,), dev, "cu_new"),
              _arg(slots, i32, (max_tokens,), dev, "slots"), _stream_on(stream, dev)), "dsa_pages_update")


def _write_args(k, v, slots, k_cache, dev):
    """What the cache writes share: (tokens, heads, dim), pages, and the arguments up to num_pages."""
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise TypeError("k: expected a 3-D tensor")
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise TypeError("k_cache: expected a 4-D tensor")
    T, K, D = shape = k.shape
    P = k_cache.shape[0]
    kp, ldk = _heads_arg(k, shape, dev, "k")
    vp, ldv = _heads_arg(v, shape, dev, "v")
    return (T, K, D, kp, ldk, vp, ldv, _arg(slots, torch.int32, (T,), dev, "slots"), P), (P, K, PAGE_SIZE, D)


def dsa_kv_write(k, v, slots, k_cache, v_cache, stream=None):
    """Keys and values ``k``, ``v`` bf16 [tokens, K, D] (rows may be strided, e.g. columns of one
    projection) to the cache rows ``slots`` (int32; -1: none) of ``k_cache``, ``v_cache`` bf16
    [num_pages, K, 64, D]; see include/dsa.h."""
    fn, dev, bf16 = lib().dsa_kv_write, torch.cuda.current_device(), torch.bfloat16
    args, shape = _write_args(k, v, slots, k_cache, dev)
    _check(fn(*args, _arg(k_cache, bf16, shape, dev, "k_cache"), _arg(v_cache, bf16, shape, dev, "v_cache"),
              _stream_on(stream, dev)), "dsa_kv_write")


def dsa_kv_write_fp8(k, v, slots, k8, k_scale, v8, v_scale, stream=None):
    """dsa_kv_write into FP8 caches: ``k8``, ``v8`` E4M3 codes as uint8 [num_pages, K, 64, 128], ``k_scale``,
    ``v_scale`` float32 [num_pages, K, 64]."""
    fn, dev, u8, f32 = lib().dsa_kv_write_fp8, torch.cuda.current_device(), torch.uint8, torch.float32
    args, shape = _write_args(k, v, slots, k8, dev)
    _check(fn(*args, _arg(k8, u8, shape, dev, "k8"), _arg(k_scale, f32, shape[:3], dev, "k_scale"),
              _arg(v8, u8, shape, dev, "v8"), _arg(v_scale, f32, shape[:3], dev, "v_scale"),
              _stream_on(stream, dev)), "dsa_kv_write_fp8")


def dsa_gqa_decode_workspace_bytes(desc, kv_heads, dim) -> int:
    return int(lib().dsa_gqa_decode_workspace_bytes(ctypes.byref(desc), kv_heads, dim))


def _grouped_shape(desc, cache, name):
    """(kv_heads, dim) of a cache [num_pages, kv_heads, 64, dim], and its shape."""
    if not isinstance(cache, torch.Tensor) or cache.dim() != 4:
        raise TypeError(f"{name}: expected a 4-D tensor")
    K, D = cache.shape[1], cache.shape[3]
    return K, D, (desc.num_pages, K, PAGE_SIZE, D)


def dsa_gqa_decode(desc, q, k, v, out, ws, sm_scale, lse=None, stream=None):
    """Attention of a decode step's queries ``q`` bf16 [T, H, D] over the paged caches ``k``, ``v`` bf16
    [num_pages, K, 64, D] of a layer with grouped heads: ``out`` bf16 [T, H, D], ``lse`` float32 [T, H] or
    None; see include/dsa.h."""
    fn, dev, bf16 = lib().dsa_gqa_decode, torch.cuda.current_device(), torch.bfloat16
    T, H = desc.batch * desc.q_per_req, desc.num_heads
    K, D, shape = _grouped_shape(desc, k, "k")
    _check(fn(ctypes.byref(desc), K, D, _arg(q, bf16, (T, H, D), dev, "q"), _arg(k, bf16, shape, dev, "k"),
              _arg(v, bf16, shape, dev, "v"), sm_scale, _arg(out, bf16, (T, H, D), dev, "out"),
              _arg(lse, torch.float32, (T, H), dev, "lse"), _arg(ws, torch.uint8, (ws.numel(),), dev, "ws"),
              ws.numel(), _stream_on(stream, dev)), "dsa_gqa_decode")


def dsa_gqa_decode_fp8kv(desc, q, k8, k_scale, v8, v_scale, out, ws, sm_scale, lse=None, stream=None):
    """dsa_gqa_decode over the FP8 caches of dsa_kv_write_fp8."""
    fn, dev, bf16 = lib().dsa_gqa_decode_fp8kv, torch.cuda.current_device(), torch.bfloat16
    u8, f32 = torch.uint8, torch.float32
    T, H = desc.batch * desc.q_per_req, desc.num_heads
    K, D, shape = _grouped_shape(desc, k8, "k8")
    _check(fn(ctypes.byref(desc), K, D, _arg(q, bf16, (T, H, D), dev, "q"), _arg(k8, u8, shape, dev, "k8"),
              _arg(k_scale, f32, shape[:3], dev, "k_scale"), _arg(v8, u8, shape, dev, "v8"),
              _arg(v_scale, f32, shape[:3], dev, "v_scale"), sm_scale, _arg(out, bf16, (T, H, D), dev, "out"),
              _arg(lse, f32, (T, H), dev, "lse"), _arg(ws, u8, (ws.numel(),), dev, "ws"), ws.numel(),
              _stream_on(stream, dev)), "dsa_gqa_decode_fp8kv")


def dsa_gqa_prefill(q, k, v, cu_q, cu_k, out, max_q, sm_scale, causal=True, lse=None, stream=None):
    """Attention of packed prompts with grouped heads: ``q`` [total_q, H, D], ``k``, ``v`` [total_k, K, D]
    (rows may be strided: columns of one projection), ``out`` [total_q, H, D], all bf16; see
    include/dsa.h."""
    fn, dev, bf16, i32 = lib().dsa_gqa_prefill, torch.cuda.current_device(), torch.bfloat16, torch.int32
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise TypeError("q, k: expected 3-D tensors")
    if not isinstance(cu_q, torch.Tensor) or cu_q.dim() != 1 or cu_q.shape[0] < 2:
        raise TypeError("cu_q: expected a 1-D tensor of at least two offsets")
    (Tq, H, D), (Tk, K, _), B1 = q.shape, k.shape, cu_q.shape[0]
    qp, ldq = _heads_arg(q, (Tq, H, D), dev, "q")
    kp, ldk = _heads_arg(k, (Tk, K, D), dev, "k")
    vp, ldv = _heads_arg(v, (Tk, K, D), dev, "v")
    _check(fn(B1 - 1, H, K, D, Tq, Tk, max_q, _arg(cu_q, i32, (B1,), dev, "cu_q"),
              _arg(cu_k, i32, (B1,), dev, "cu_k"), qp, ldq, kp, ldk, vp, ldv, sm_scale, 1 if causal else 0,
              _arg(out, bf16, (Tq, H, D), dev, "out"), _arg(lse, torch.float32, (Tq, H), dev, "lse"),
              _stream_on(stream, dev)), "dsa_gqa_prefill")


def dsa_rmsnorm(x, weight, eps, residual=None, residual_out=None, y=None, y8=None, y_scale=None,
                group=128, stream=None):
    """Residual addition and root-mean-square norm of ``x`` [rows, dim] (rows may be strided, e.g. a
    slice of a wider projection), into ``y`` (bf16) and / or ``y8`` + ``y_scale`` (E4M3 codes as uint8,
    fp32 scales [rows, ceil(dim / 128)], or [rows, 1] for ``group=0``); see include/dsa.h."""
    fn, dev, bf16 = lib().dsa_rmsnorm, torch.cuda.current_device(), torch.bfloat16
    xp, ld = _rows_arg(x, bf16, dev, "x")
    shape = x.shape
    rows, dim = shape
    _check(fn(rows, dim, xp, ld, _arg(residual, bf16, shape, dev, "residual"),
              _arg(weight, bf16, (dim,), dev, "weight"), eps, group,
              _arg(residual_out, bf16, shape, dev, "residual_out"), _arg(y, bf16, shape, dev, "y"),
              _arg(y8, torch.uint8, shape, dev, "y8"),
              _arg(y_scale, torch.float32, (rows, -(-dim // 128) if group else 1), dev, "y_scale"),
              _stream_on(stream, dev)), "dsa_rmsnorm")


def dsa_decode_mli(desc, q_fp8, q_scale, w, k_fp8, k_scale, q, kv, topk_prev, topk_next, out, ws,
                   max_seqlen, sm_scale, num_splits=0, stream=None):
    """One layer of the Multi-layer Indexer schedule: attention over
    ``topk_prev`` while this layer's indexer and top-k write ``topk_next``
    (see include/dsa.h)."""
    _check(lib().dsa_decode_mli(
        ctypes.byref(desc), _ptr(q_fp8, torch.uint8, "q_fp8"), _ptr(q_scale, torch.float32, "q_scale"),
        _ptr(w, torch.float32, "w"), _ptr(k_fp8, torch.uint8, "k_fp8"),
        _ptr(k_scale, torch.float32, "k_scale"), _u16(q, "q"), _u16(kv, "kv"),
        _ptr(topk_prev, torch.int32, "topk_prev"), _ptr(topk_next, torch.int32, "topk_next"),
        float(sm_scale), int(num_splits), int(max_seqlen), _ptr(out, torch.float32, "out"),
        _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)), "dsa_decode_mli")


def dsa_num_splits_mli(desc) -> int:
    return int(lib().dsa_num_splits_mli(ctypes.byref(desc)))


def dsa_step_layout_get(batch, q_per_req, num_heads, max_pages) -> StepLayout:
    lay = StepLayout()
    _check(lib().dsa_step_layout_get(int(batch), int(q_per_req), int(num_heads), int(max_pages),
                                     ctypes.byref(lay)), "dsa_step_layout_get")
    return lay


def step_views(block: torch.Tensor, layout: StepLayout, batch, q_per_req, num_heads, max_pages):
    """Typed views of each step input inside a uint8 block (host or device)
    laid out by ``dsa_step_layout_get``."""
    if block.dtype != torch.uint8 or block.dim() != 1 or block.numel() < layout.bytes:
        raise ValueError("block must be a 1-D uint8 tensor of at least layout.bytes")
    T = int(batch) * int(q_per_req)
    parts = (("q_fp8", torch.uint8, (T, 64, 128)), ("q_scale", torch.float32, (T,)),
             ("w", torch.float32, (T, 64)), ("q", torch.bfloat16, (T, int(num_heads), 576)),
             ("seqlens", torch.int32, (int(batch),)),
             ("page_table", torch.int32, (int(batch), int(max_pages))))
    views = {}
    for name, dtype, shape in parts:
        off = getattr(layout, name)
        n = 1
        for x in shape:
            n *= x
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        views[name] = block[off:off + nbytes].view(dtype).view(shape)
    return views


class HostStepPipeline:
    """Decode layers whose per-step inputs start in host memory and whose
    outputs end there, with the copies of one step overlapping the layers of
    its neighbours: the resources of a ``dsa_decode_step_ring`` (two device
    input blocks laid out by ``dsa_step_layout_get``, two device outputs, the
    workspace, a copy-in and a copy-out stream, six events), and one library
    call per step.  Step i (slot i % 2) copies its block in once the layer of
    step i - 2 is done reading that slot, its layer waits for that copy and
    for the output copy of step i - 2, and its output is copied out after its
    layer; so while layer i runs, the inputs of step i + 1 come in and the
    output of step i - 1 goes out.  The caches and the workspace stay in
    device memory.  A host block may be rewritten once the copy of the step
    that read it is done (``input_copied(i)``); ``host_out`` of step i is
    valid once ``output_copied(i)`` (or ``drain``) has been waited on.  Every
    step of one pipeline runs its layer on the same stream (the steps share
    one workspace); another stream raises.
    """

    def __init__(self, batch, q_per_req, num_heads, topk, max_pages, num_pages, max_seqlen,
                 sm_scale, num_splits=0, device=None):
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        self.layout = dsa_step_layout_get(batch, q_per_req, num_heads, max_pages)
        self.dims = (batch, q_per_req, num_heads, max_pages)
        self.dev_in = [torch.empty(self.layout.bytes, dtype=torch.uint8, device=device)
                       for _ in range(2)]
        self.views = [step_views(d, self.layout, *self.dims) for d in self.dev_in]
        T = batch * q_per_req
        self.out = [torch.empty((T, num_heads, 512), dtype=torch.float32, device=device)
                    for _ in range(2)]
        self.desc = make_desc(self.views[0]["seqlens"], self.views[0]["page_table"], q_per_req,
                              num_heads, topk, num_pages)
        self.splits = num_splits if num_splits else dsa_num_splits_auto(self.desc)
        self.ws = torch.empty(dsa_workspace_bytes(self.desc, max_seqlen, self.splits),
                              dtype=torch.uint8, device=device)
        self.max_seqlen, self.sm_scale = int(max_seqlen), float(sm_scale)
        self.h2d = torch.cuda.Stream(device)
        self.d2h = torch.cuda.Stream(device)
        mk = lambda: [torch.cuda.Event() for _ in range(2)]
        self.ev_in, self.ev_done, self.ev_out = mk(), mk(), mk()
        with torch.cuda.device(device):
            for e in self.ev_in + self.ev_done + self.ev_out:
                e.record()   # creates the event (torch creates them on first record)
            torch.cuda.current_stream().synchronize()
        r = StepRing()
        for b in range(2):
            r.dev_in[b] = _ptr(self.dev_in[b], torch.uint8, "dev_in")
            r.out[b] = _ptr(self.out[b], torch.float32, "out")
            r.ev_in[b], r.ev_done[b], r.ev_out[b] = (self.ev_in[b].cuda_event,
                                                     self.ev_done[b].cuda_event,
                                                     self.ev_out[b].cuda_event)
        r.ws, r.ws_bytes = _ptr(self.ws, torch.uint8, "ws"), self.ws.numel()
        r.copy_in_stream, r.copy_out_stream = self.h2d.cuda_stream, self.d2h.cuda_stream
        r.step = 0
        self.ring = r
        self._ring_fn = lib().dsa_decode_step_ring
        self._calls = {}
        self._stream = None

    @property
    def steps(self) -> int:
        return int(self.ring.step)

    def submit(self, host_in, host_out, k_fp8, k_scale, kv, stream=None):
        """Queues one step: host_in (a pinned uint8 block) -> layer over the
        given caches -> host_out (pinned float32 [T, H, 512])."""
        comp = torch.cuda.current_stream() if stream is None else stream
        sid = _stream(comp)
        if self._stream is None:
            self._stream = sid
        elif sid != self._stream:
            raise ValueError("every step of a HostStepPipeline runs on the same stream")
        # The call's arguments are checked and packed once per host buffer
        # pair, cache set and stream; later steps only issue the call.
        key = (host_in.data_ptr(), host_out.data_ptr(), k_fp8.data_ptr(), k_scale.data_ptr(),
               kv.data_ptr(), k_fp8.dtype, k_scale.dtype, kv.dtype, sid)
        args = self._calls.get(key)
        if args is None:
            if host_in.dtype != torch.uint8 or host_in.is_cuda or host_in.numel() < self.layout.bytes:
                raise ValueError("host_in: a host uint8 block of at least layout.bytes")
            if host_out.is_cuda or host_out.dtype != torch.float32 or host_out.shape != self.out[0].shape:
                raise ValueError("host_out: a host float32 tensor shaped like the output")
            args = (ctypes.byref(self.desc), ctypes.byref(self.ring),
                    _host_ptr(host_in, torch.uint8, "host_in"),
                    _host_ptr(host_out, torch.float32, "host_out"),
                    _ptr(k_fp8, torch.uint8, "k_fp8"), _ptr(k_scale, torch.float32, "k_scale"),
                    _u16(kv, "kv"), self.sm_scale, self.splits, self.max_seqlen, sid)
            self._calls[key] = args
        _check(self._ring_fn(*args), "dsa_decode_step_ring")

    def input_copied(self, step):
        """Event after which the host block of `step` may be rewritten (valid
        until step + 2 is submitted)."""
        return self.ev_in[step % 2]

    def output_copied(self, step):
        """Event after which host_out of `step` holds its output (valid until
        step + 2 is submitted)."""
        return self.ev_out[step % 2]

    def drain(self, stream=None):
        """Makes `stream` (default: the current one) wait for every queued copy."""
        comp = torch.cuda.current_stream() if stream is None else stream
        comp.wait_stream(self.h2d)
        comp.wait_stream(self.d2h)


def _host_ptr(t, dtype, name):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.is_cuda:
        raise ValueError(f"{name}: expected a host tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def dsa_decode_step_host(desc, host_in, dev_in, k_fp8, k_scale, kv, out, host_out, ws, max_seqlen,
                         sm_scale, num_splits=0, stream=None):
    """One decode layer from a host input block to a host output (see
    include/dsa.h): one host-to-device copy, the fused layer, one
    device-to-host copy, all queued on ``stream``."""
    _check(lib().dsa_decode_step_host(
        ctypes.byref(desc), _host_ptr(host_in, torch.uint8, "host_in"),
        _ptr(dev_in, torch.uint8, "dev_in"), _ptr(k_fp8, torch.uint8, "k_fp8"),
        _ptr(k_scale, torch.float32, "k_scale"), _u16(kv, "kv"), float(sm_scale),
        int(num_splits), int(max_seqlen), _ptr(out, torch.float32, "out"),
        _host_ptr(host_out, torch.float32, "host_out"), _ptr(ws, torch.uint8, "ws"), ws.numel(),
        _stream(stream)), "dsa_decode_step_host")


def dsa_get_device_error(stream=None) -> int:
    return int(lib().dsa_get_device_error(_stream(stream)))


def dsa_status_str(status: int) -> str:
    return lib().dsa_status_str(int(status)).decode()


def dsa_version() -> str:
    return lib().dsa_version().decode()


def dsa_debug_set_wait_cycles(cycles: int):
    """Bound of the indexer's pipeline waits in SM cycles (0: the default);
    a test hook for the timeout path (see include/dsa.h)."""
    _check(lib().dsa_debug_set_wait_cycles(int(cycles)), "dsa_debug_set_wait_cycles")


# ---------------------------------------------------------------------------
# Convenience layer over a synthetic ``workloads.Workload`` (allocates outputs
# with torch, then calls the ABI above).
# ---------------------------------------------------------------------------

def workload_desc(wl) -> DecodeDesc:
    s = wl.spec
    return make_desc(wl.seqlens, wl.page_table, s.q_per_req, s.num_heads, s.topk, wl.num_pages)


def logits_ld(wl) -> int:
    return wl.max_pages * PAGE_SIZE


def run_indexer(wl, layer: int = 0, stream=None) -> torch.Tensor:
    lc = wl.layers[layer]
    T = wl.spec.num_tokens
    ld = logits_ld(wl)
    logits = torch.full((T, ld), float("nan"), device=wl.q_fp8.device, dtype=torch.float32)
    dsa_indexer_logits(workload_desc(wl), wl.q_fp8, wl.q_scale, wl.w, lc.k_fp8, lc.k_scale,
                       logits, ld, stream)
    return logits


def run_topk(wl, logits: torch.Tensor, stream=None) -> torch.Tensor:
    desc = workload_desc(wl)
    ld = int(logits.shape[1])
    ws = torch.empty(dsa_topk_workspace_bytes(desc, ld), dtype=torch.uint8, device=logits.device)
    out = torch.empty((wl.spec.num_tokens, wl.spec.topk), dtype=torch.int32, device=logits.device)
    dsa_topk(desc, logits, out, ws, ld, stream)
    return out


def run_sparse_mla_split(wl, topk_idx, num_splits=0, layer: int = 0, stream=None):
    lc = wl.layers[layer]
    desc = workload_desc(wl)
    S = dsa_num_splits_auto(desc) if num_splits == 0 else num_splits
    T, H = wl.spec.num_tokens, wl.spec.num_heads
    mid_o = torch.empty((T, H, S, 512), dtype=torch.float32, device=lc.q.device)
    mid_lse = torch.empty((T, H, S), dtype=torch.float32, device=lc.q.device)
    dsa_sparse_mla_decode_split(desc, lc.q, lc.kv, topk_idx, S, wl.spec.sm_scale, mid_o, mid_lse,
                                stream)
    return mid_o, mid_lse


def run_merge(mid_o, mid_lse, stream=None):
    T, H, S, _ = mid_o.shape
    out = torch.empty((T, H, 512), dtype=torch.float32, device=mid_o.device)
    lse = torch.empty((T, H), dtype=torch.float32, device=mid_o.device)
    dsa_merge(T * H, S, mid_o, mid_lse, out, lse, stream)
    return out, lse


def alloc_workspace(wl, num_splits=0) -> torch.Tensor:
    desc = workload_desc(wl)
    n = dsa_workspace_bytes(desc, wl.max_seqlen, num_splits)
    return torch.empty(n, dtype=torch.uint8, device=wl.q_fp8.device)


def run_decode(wl, ws=None, num_splits=0, layer: int = 0, topk_in=None, topk_out=None,
               out=None, stream=None, stage_events=None) -> torch.Tensor:
    lc = wl.layers[layer]
    T, H = wl.spec.num_tokens, wl.spec.num_heads
    if ws is None:
        ws = alloc_workspace(wl, num_splits)
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.float32, device=lc.q.device)
    dsa_decode_fused(workload_desc(wl), wl.q_fp8, wl.q_scale, wl.w, lc.k_fp8, lc.k_scale, lc.q,
                     lc.kv, out, ws, wl.max_seqlen, wl.spec.sm_scale, num_splits, topk_in,
                     topk_out, stream, stage_events)
    return out
