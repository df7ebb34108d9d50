"""Thin Python binding of the kvpool C ABI (``include/kvpool.h``).

Argument marshalling only: torch tensors are passed as raw device pointers,
the current (or given) torch CUDA stream as a ``cudaStream_t``.  Every step of
the path runs in the CUDA kernels of ``libkvpool.so``; there is no CPU or
PyTorch fallback -- if the library cannot be built or loaded this module
raises.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
from dataclasses import dataclass, field
from typing import Optional, Sequence

import numpy as np

F32, BF16, FP8_E4M3, FP4_E2M1 = 0, 1, 2, 3  # FP4: indexer entries only (PoolConfig.idx_fp4)
SWA_ONLY, CSA, HCA, CSA_HCA = 0, 1, 2, 3
FLAG_NO_DEVICE = 1
OK, ERR_INVALID_ARG, ERR_OUT_OF_BLOCKS, ERR_OUT_OF_REQUESTS, ERR_BAD_REQUEST = 0, -1, -2, -3, -4
ERR_NOT_SHAREABLE, ERR_CUDA, ERR_DEVICE_CHECK, ERR_CAPACITY, ERR_BAD_IMAGE = -5, -6, -7, -8, -9
KERNEL_APPEND, KERNEL_SCORE, KERNEL_SELECT, KERNEL_ATTEND, KERNEL_COMBINE, KERNEL_IMAGE = range(6)
KERNEL_NAMES = ["append", "score", "select", "attend", "combine", "image"]
IMAGE_WINDOW = 1  # prefix image flag: include the SWA window (a checkpoint)
PROFILE_COUNT = 1 << 16  # profiling flag: count launches and bytes without events

EXPORTS = ["kvpool_required_bytes", "kvpool_create", "kvpool_destroy", "kvpool_alloc_request",
           "kvpool_free_request", "kvpool_share_prefix", "kvpool_append", "kvpool_decode_attend",
           "kvpool_request_info", "kvpool_block_refcount", "kvpool_free_block_count", "kvpool_get_layout",
           "kvpool_check_device", "kvpool_profile_enable", "kvpool_profile_read", "kvpool_last_error",
           "kvpool_topk_static", "kvpool_profile_timeline", "kvpool_fingerprint", "kvpool_image_bytes",
           "kvpool_export_prefix", "kvpool_import_prefix", "kvpool_host_slot_bytes", "kvpool_set_host_pool",
           "kvpool_offload", "kvpool_fetch", "kvpool_block_location", "kvpool_epoch", "kvpool_block_activity",
           "kvpool_inactive_blocks", "kvpool_wait_selftest", "kvpool_topk_static_check", "kvpool_rope_table",
           "kvpool_qk_norm_rope", "kvpool_window_workspace", "kvpool_window_attend",
           "kvpool_decode_attend_shared", "kvpool_window_check", "kvpool_set_share_bytes", "kvpool_qk_norm_rope_axes",
           "kvpool_kv4_page_bytes", "kvpool_kv4_store", "kvpool_kv4_load", "kvpool_kv4_workspace", "kvpool_kv4_attend",
           "kvpool_kv4_evict"]


class KvpoolError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"kvpool error {code}: {msg}")
        self.code = code


class _Config(C.Structure):
    _fields_ = [("m", C.c_int32), ("m_prime", C.c_int32), ("n_win", C.c_int32), ("heads", C.c_int32),
                ("head_dim", C.c_int32), ("idx_heads", C.c_int32), ("idx_dim", C.c_int32),
                ("in_dtype", C.c_int32), ("cache_dtype", C.c_int32), ("n_layers", C.c_int32),
                ("layer_kinds", C.POINTER(C.c_int32)), ("max_requests", C.c_int32), ("max_blocks", C.c_int32),
                ("max_blocks_per_request", C.c_int32), ("max_batch", C.c_int32), ("max_top_k", C.c_int32),
                ("gate_csa", C.POINTER(C.c_float)), ("gate_hca", C.POINTER(C.c_float)),
                ("gate_idx", C.POINTER(C.c_float)), ("flags", C.c_uint32), ("idx_fp4", C.c_int32),
                ("csa_hot_slots", C.c_int32), ("csa_host_slots", C.c_int32), ("idx_per_token", C.c_int32)]


class _Info(C.Structure):
    _fields_ = [("length", C.c_int64), ("n_csa", C.c_int64), ("n_hca", C.c_int64), ("csa_tail", C.c_int32),
                ("hca_tail", C.c_int32), ("n_blocks", C.c_int32), ("window", C.c_int32)]


class _Layout(C.Structure):
    _fields_ = [("entry_bytes", C.c_int64), ("idx_entry_bytes", C.c_int64), ("csa_per_block", C.c_int32),
                ("staging_base", C.c_int32), ("table_offset", C.c_int64), ("error_offset", C.c_int64),
                ("total_bytes", C.c_int64), ("csa_staging_base", C.c_int32), ("csa_hot_slots", C.c_int32),
                ("host_slot_bytes", C.c_int64), ("csa_loc_offset", C.c_int64), ("activity_offset", C.c_int64)]


class _LayerLayout(C.Structure):
    _fields_ = [("kind", C.c_int32), ("pad", C.c_int32), ("csa_offset", C.c_int64), ("csa_block_bytes", C.c_int64),
                ("idx_offset", C.c_int64), ("idx_block_bytes", C.c_int64), ("idx_scale_offset", C.c_int64),
                ("hca_offset", C.c_int64), ("hca_block_bytes", C.c_int64), ("ring_offset", C.c_int64),
                ("ring_request_bytes", C.c_int64), ("acc_offset", C.c_int64), ("acc_request_bytes", C.c_int64),
                ("csa_host_offset", C.c_int64)]


_lib = None


def lib():
    """Load libkvpool.so (building it in-tree first if it is missing or stale)."""
    global _lib
    if _lib is None:
        from ._build import build_lib
        path = build_lib("kvpool")
        L = C.CDLL(path)
        vp, i32, i64 = C.c_void_p, C.c_int32, C.c_int64
        L.kvpool_required_bytes.restype = C.c_size_t
        L.kvpool_required_bytes.argtypes = [C.POINTER(_Config)]
        L.kvpool_create.argtypes = [C.POINTER(_Config), vp, C.c_size_t, vp, C.POINTER(vp)]
        L.kvpool_destroy.argtypes = [vp]
        L.kvpool_alloc_request.argtypes = [vp, C.POINTER(i32)]
        L.kvpool_free_request.argtypes = [vp, i32]
        L.kvpool_share_prefix.argtypes = [vp, i32, i32, i64, vp, vp, vp]
        L.kvpool_append.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp]
        L.kvpool_decode_attend.argtypes = [vp, i32, i32, vp, vp, vp, i32, vp, vp, vp]
        L.kvpool_decode_attend_shared.argtypes = [vp, i32, i32, vp, i64, vp, vp, i32, vp, vp, vp]
        L.kvpool_set_share_bytes.argtypes = [vp, i64]
        L.kvpool_request_info.argtypes = [vp, i32, C.POINTER(_Info), vp, i32]
        L.kvpool_block_refcount.argtypes = [vp, i32]
        L.kvpool_free_block_count.argtypes = [vp]
        L.kvpool_get_layout.argtypes = [vp, C.POINTER(_Layout), i32, C.POINTER(_LayerLayout)]
        L.kvpool_check_device.argtypes = [vp, vp, C.POINTER(C.c_uint32)]
        L.kvpool_profile_enable.argtypes = [vp, C.c_int]
        L.kvpool_profile_read.argtypes = [vp, i32, C.POINTER(C.c_double), C.POINTER(i64), C.POINTER(i64)]
        L.kvpool_topk_static.argtypes = [vp, i32, i32, i32, vp, vp]
        L.kvpool_topk_static_check.argtypes = [vp, C.POINTER(C.c_uint32)]
        L.kvpool_profile_timeline.argtypes = [vp, i32, vp]
        L.kvpool_fingerprint.restype = C.c_uint64
        L.kvpool_fingerprint.argtypes = [vp]
        L.kvpool_image_bytes.restype = i64
        L.kvpool_image_bytes.argtypes = [vp, i64, C.c_uint32]
        L.kvpool_export_prefix.argtypes = [vp, i32, i64, C.c_uint32, vp, i64, vp]
        L.kvpool_import_prefix.argtypes = [vp, i32, vp, i64, vp, vp, vp]
        L.kvpool_host_slot_bytes.restype = i64
        L.kvpool_host_slot_bytes.argtypes = [vp]
        L.kvpool_set_host_pool.argtypes = [vp, vp, i64]
        L.kvpool_offload.argtypes = [vp, i32, vp, vp]
        L.kvpool_fetch.argtypes = [vp, i32, vp, vp]
        L.kvpool_block_location.argtypes = [vp, i32, C.POINTER(i32)]
        L.kvpool_epoch.restype = C.c_uint32
        L.kvpool_epoch.argtypes = [vp]
        L.kvpool_block_activity.argtypes = [vp, i32, vp, vp, vp]
        L.kvpool_inactive_blocks.restype = i32
        L.kvpool_inactive_blocks.argtypes = [vp, C.c_uint32, vp, i32, vp]
        L.kvpool_wait_selftest.argtypes = [vp, vp]
        L.kvpool_rope_table.argtypes = [i32, vp, vp]
        cp = C.c_char_p  # a packed structure
        L.kvpool_qk_norm_rope.argtypes = [i32, i32, i64, cp, cp, cp, cp, vp, vp, C.c_float, i32, i32, vp, vp, vp]
        L.kvpool_qk_norm_rope_axes.argtypes = L.kvpool_qk_norm_rope.argtypes[:-1] + [i32, cp, vp]
        L.kvpool_window_workspace.restype = i64
        L.kvpool_window_workspace.argtypes = [cp, i32, vp, vp, vp]
        L.kvpool_window_attend.argtypes = [cp, i32, vp, vp, vp, vp, i64, vp]
        L.kvpool_window_check.argtypes = [vp, C.POINTER(C.c_uint32)]
        L.kvpool_kv4_page_bytes.restype = i64
        L.kvpool_kv4_page_bytes.argtypes = [i32, i32, i32]
        L.kvpool_kv4_store.argtypes = L.kvpool_kv4_load.argtypes = [cp, i32, cp, cp, i64, i32, vp, vp, vp]
        L.kvpool_kv4_workspace.restype = i64
        L.kvpool_kv4_workspace.argtypes = [cp, i32, vp, vp]
        L.kvpool_kv4_attend.argtypes = [cp, i32, vp, vp, vp, i64, vp]
        L.kvpool_kv4_evict.argtypes = [cp, i32, vp, vp]
        L.kvpool_last_error.restype = C.c_char_p
        L.kvpool_last_error.argtypes = [vp]
        _lib = L
    return _lib


def library_path() -> str:
    return lib()._name


@dataclass
class PoolConfig:
    m: int
    m_prime: int
    n_win: int
    heads: int
    head_dim: int
    idx_heads: int
    idx_dim: int
    in_dtype: int
    cache_dtype: int
    layer_kinds: Sequence[int]
    max_requests: int
    max_blocks: int
    max_blocks_per_request: int
    max_batch: int
    max_top_k: int
    gate_csa: np.ndarray  # [n_layers][heads][m] logits
    gate_hca: np.ndarray  # [n_layers][heads][m_prime]
    gate_idx: np.ndarray  # [n_layers][idx_heads][m]
    flags: int = 0
    idx_fp4: int = 0  # 1: indexer entries in FP4 (e2m1 + one bf16 scale)
    csa_hot_slots: int = 0  # HiSparse: GPU slots for sealed blocks' CSA entries (0 = off)
    csa_host_slots: int = 0  # HiSparse: host slots for offloaded CSA entries
    idx_per_token: int = 0  # 1: one indexer key per token (128 per block) instead of one per CSA entry
    _keep: list = field(default_factory=list, repr=False)

    def to_c(self) -> _Config:
        kinds = np.ascontiguousarray(self.layer_kinds, dtype=np.int32)
        g = [np.ascontiguousarray(x, dtype=np.float32).reshape(-1) for x in (self.gate_csa, self.gate_hca,
                                                                             self.gate_idx)]
        self._keep = [kinds] + g
        fp = C.POINTER(C.c_float)
        return _Config(self.m, self.m_prime, self.n_win, self.heads, self.head_dim, self.idx_heads, self.idx_dim,
                       self.in_dtype, self.cache_dtype, kinds.size, kinds.ctypes.data_as(C.POINTER(C.c_int32)),
                       self.max_requests, self.max_blocks, self.max_blocks_per_request, self.max_batch,
                       self.max_top_k, g[0].ctypes.data_as(fp), g[1].ctypes.data_as(fp), g[2].ctypes.data_as(fp),
                       self.flags, self.idx_fp4, self.csa_hot_slots, self.csa_host_slots, self.idx_per_token)


def required_bytes(cfg: PoolConfig) -> int:
    c = cfg.to_c()
    return int(lib().kvpool_required_bytes(C.byref(c)))


def topk_static(scores, top_k: int, out, stream=None) -> int:
    """Top-k of each row of a [n_rows][n_cols] fp32 device tensor into
    ``out`` ([n_rows][top_k] int32) using only the library's static device
    scratch (no allocation); see kvpool_topk_static in include/kvpool.h.
    Raises ValueError for tensors the kernels cannot take as they are."""
    import torch
    if scores.dim() != 2 or scores.dtype != torch.float32 or not scores.is_cuda or not scores.is_contiguous():
        raise ValueError("topk_static: scores must be a contiguous 2-D float32 CUDA tensor")
    n_rows, n_cols = scores.shape
    if (out.dtype != torch.int32 or not out.is_cuda or not out.is_contiguous() or out.device != scores.device
            or tuple(out.shape) != (n_rows, top_k)):
        raise ValueError("topk_static: out must be a contiguous int32 [n_rows][top_k] tensor on the scores' device")
    return lib().kvpool_topk_static(scores.data_ptr(), n_rows, n_cols, top_k, out.data_ptr(), _stream(stream))


def topk_static_check(stream=None) -> tuple:
    """(return code, device error flags) of the last topk_static call on the
    current device; synchronizes the stream."""
    w = C.c_uint32(0)
    rc = lib().kvpool_topk_static_check(_stream(stream), C.byref(w))
    return int(rc), int(w.value)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:  # the current device's current stream
        from torch import _C
        return _C._cuda_getCurrentRawStream(_C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _host_buffer(x):
    """(address, bytes) of a host buffer: a numpy array or a CPU torch tensor."""
    if isinstance(x, np.ndarray):
        return x.ctypes.data, x.nbytes
    return x.data_ptr(), x.numel() * x.element_size()


def _i32(a) -> np.ndarray:
    if type(a) is np.ndarray and a.dtype == np.int32 and a.flags.c_contiguous:
        return a
    return np.ascontiguousarray(a, dtype=np.int32)


def _dtype(t) -> int:
    import torch
    if t.dtype is torch.bfloat16:
        return BF16
    if t.dtype is torch.float32:
        return F32
    raise ValueError("tensors must be float32 or bfloat16")


# kvpool_heads and kvpool_window_args of include/kvpool.h, packed in one go
# (filling ctypes structures field by field takes longer than a small launch)
_HEADS = struct.Struct("@Pqqii")
_WINDOW_ARGS = struct.Struct("@ii" + 4 * "Pqqii" + "qqPiifi")
_KV4 = struct.Struct("@PqPqiiiiiffi")  # kvpool_kv4
_KV4_ARGS = struct.Struct("@if" + 2 * "Pqqii" + "qPPqqfi")  # kvpool_kv4_args behind its cache
_KV4_EVICT = struct.Struct("@PqiiPqqPqqPiiii")  # kvpool_kv4_evict_args behind its cache


def _rows(t, what: str, like=None, out: bool = False) -> tuple:
    """The kvpool_heads fields of a [tokens][heads][dim] CUDA tensor."""
    shape = t.shape
    if len(shape) != 3 or not t.is_cuda:
        raise ValueError(f"{what} must be a [tokens][heads][dim] CUDA tensor")
    n, heads, dim = shape
    size = 2
    if like is not None:
        if t.dtype is not like[0] or dim != like[1] or t.get_device() != like[2]:
            raise ValueError(f"{what} must have the type, head dim and device of the other tensors")
        size = like[3]
    ts, hs, vs = t.stride()
    # the stride of an axis of length 1 is never used
    if n <= 1:
        ts = 0
    if heads <= 1:
        hs = 0
    ptr = t.data_ptr()
    if (ptr | ts * size | hs * size) & 15 and n * heads * dim or vs != 1 and dim > 1:
        raise ValueError(f"{what}: a head's values must be adjacent, data and strides whole multiples of 16 bytes")
    if out and (n > 1 and ts < dim or heads > 1 and hs < dim or
                n > 1 and heads > 1 and (hs < ts * (n - 1) + dim if ts < hs else ts < hs * (heads - 1) + dim)):
        raise ValueError(f"{what}: two values share a place")
    return ptr, ts, hs, heads, 0


def _like(t) -> tuple:
    """What _rows compares the other tensors of a call with."""
    return t.dtype, t.shape[-1], t.get_device(), t.element_size()


def _stream_of(stream, index: int) -> int:
    """The given stream, or the device's current one."""
    if stream is None:
        from torch import _C
        return _C._cuda_getCurrentRawStream(index)
    return _stream(stream)


def _fresh(t, stream, raw: int):
    """An uninitialized contiguous tensor like t whose memory belongs to
    `stream`, the one that will write it, and its kvpool_heads fields."""
    import torch
    n, heads, dim = t.shape
    if stream is None or raw == torch._C._cuda_getCurrentRawStream(t.get_device()):
        o = torch.empty((n, heads, dim), dtype=t.dtype, device=t.device)
    else:
        with torch.cuda.stream(torch.cuda.ExternalStream(raw, device=t.device)):
            o = torch.empty((n, heads, dim), dtype=t.dtype, device=t.device)
    return o, (o.data_ptr(), heads * dim if n > 1 else 0, dim if heads > 1 else 0, heads, 0)


def _fresh_bytes(n: int, device, stream, raw: int):
    import torch
    if stream is None or raw == torch._C._cuda_getCurrentRawStream(device.index):
        return torch.empty(n, dtype=torch.uint8, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(raw, device=device)):
        return torch.empty(n, dtype=torch.uint8, device=device)


def _need(t, what: str, dtype, shape, index: int) -> int:
    """The address of a contiguous tensor of that type and shape on that device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}")
    return t.data_ptr()


def _i64(x) -> np.ndarray:
    a = x if type(x) is np.ndarray else np.asarray(x)
    if a.dtype != np.int64 or a.ndim != 1 or not a.flags.c_contiguous:
        if a.ndim != 1 or a.size and (a.dtype.kind not in "iu" or a.dtype == np.uint64):
            raise ValueError("lengths and starts must be one integer per segment")
        a = np.ascontiguousarray(a, dtype=np.int64)
    return a


def rope_table(rot_dim: int, theta: float = 10000.0, inv_freq=None, device="cuda"):
    """The rotation table of qk_norm_rope on `device`: int64 [rot_dim / 2], the
    frequencies theta ** (-2i / rot_dim) (or inv_freq, radians per position) as
    64-bit fractions of a turn; see kvpool_rope_table in include/kvpool.h."""
    import torch
    if inv_freq is None:
        inv_freq = theta ** (-np.arange(0, rot_dim, 2, dtype=np.float64) / max(rot_dim, 1))
    f = np.ascontiguousarray(inv_freq, dtype=np.float64)
    if f.shape != (rot_dim // 2,):
        raise ValueError("rope_table: inv_freq must have rot_dim / 2 values")
    out = np.empty(max(f.size, 1), np.uint64)
    rc = lib().kvpool_rope_table(rot_dim, f.ctypes.data, out.ctypes.data)
    if rc != OK:
        raise KvpoolError(rc, "rope_table: rot_dim must be a multiple of 16 up to 256, the frequencies finite")
    return torch.from_numpy(out[:f.size].view(np.int64)).to(device)


def qk_norm_rope(q, k, positions, table, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                 out_q=None, out_k=None, stream=None, axes=None):
    """Norm every head of q and k ([tokens][heads][dim], float32 or bfloat16,
    either may be None) and rotate it by its token's position (int64
    [tokens]) with the table of rope_table (None: norms only); returns (out_q,
    out_k), which may be given and may be q and k themselves.  axes: rot_dim / 2
    axis numbers (host integers); positions are then [tokens][n_axes] and pair i
    turns by the one on axis axes[i].  No gradients flow through.  See
    kvpool_qk_norm_rope and kvpool_qk_norm_rope_axes in include/kvpool.h."""
    import torch
    x = q if q is not None else k
    if x is None or not x.is_cuda:
        raise ValueError("qk_norm_rope: q or k must be a CUDA tensor")
    like = _like(x)
    index = like[2]
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return qk_norm_rope(q, k, positions, table, q_weight, k_weight, eps, interleaved, out_q, out_k, stream, axes)
    kind = _dtype(x)
    raw = _stream_of(stream, index)
    T = x.shape[0]
    qi = ki = qo = ko = None
    if q is not None:
        qi = _HEADS.pack(*_rows(q, "q", like))
        if out_q is None:
            out_q, r = _fresh(q, stream, raw)
        else:
            r = _rows(out_q, "out_q", like, True)
            if out_q.shape != q.shape:
                raise ValueError("qk_norm_rope: out_q must have the shape of q")
        qo = _HEADS.pack(*r)
    if k is not None:
        ki = _HEADS.pack(*_rows(k, "k", like))
        if k.shape[0] != T:
            raise ValueError("qk_norm_rope: q and k must have the same tokens")
        if out_k is None:
            out_k, r = _fresh(k, stream, raw)
        else:
            r = _rows(out_k, "out_k", like, True)
            if out_k.shape != k.shape:
                raise ValueError("qk_norm_rope: out_k must have the shape of k")
        ko = _HEADS.pack(*r)
    D = like[1]
    rot, tab, pos = 0, None, None
    if table is not None:
        rot = 2 * table.numel()
        tab = _need(table, "table", torch.int64, (rot // 2,), index) or None
        if axes is None:
            pos = _need(positions, "positions", torch.int64, (T,), index) or None
        else:
            if positions.dim() != 2:
                raise ValueError("qk_norm_rope: with axes, positions must be [tokens][n_axes]")
            n_axes = positions.shape[1]
            pos = _need(positions, "positions", torch.int64, (T, n_axes), index) or None
            try:
                axes = bytes(axes.tolist() if hasattr(axes, "tolist") else list(axes))
            except (TypeError, ValueError):
                raise ValueError("qk_norm_rope: axes must be small host integers") from None
            if len(axes) != rot // 2:
                raise ValueError("qk_norm_rope: axes must have one axis per pair (rot_dim / 2)")
    elif axes is not None:
        raise ValueError("qk_norm_rope: axes need a table")
    qw = None if q_weight is None else _need(q_weight, "q_weight", torch.float32, (D,), index)
    kw = None if k_weight is None else _need(k_weight, "k_weight", torch.float32, (D,), index)
    call = (kind, D, T, qi, ki, qo, ko, qw, kw, eps, rot, 1 if interleaved else 0, tab, pos)
    if axes is None:
        rc = lib().kvpool_qk_norm_rope(*call, raw)
    else:
        rc = lib().kvpool_qk_norm_rope_axes(*call, n_axes, axes, raw)
    if rc != OK:
        raise KvpoolError(rc, "qk_norm_rope refused its arguments" if rc == ERR_INVALID_ARG else "qk_norm_rope: CUDA error")
    return out_q if q is not None else None, out_k if k is not None else None


def window_attend(q, k, v, q_len, k_start, k_len, window: int, n_sink: int = 0, scale=None, out=None, lse=None,
                  workspace=None, stream=None):
    """Attention of a ragged batch over raw K/V rows with a sliding window and
    n_sink first tokens that stay visible; returns out ([rows][q heads][dim],
    like q, and q itself if given as out).  bf16 prompts round each softmax
    weight to bf16 once; fp32 tensors are fp32 throughout.  No gradients flow
    through.  q_len, k_start, k_len: host integers per segment; lse: a float32
    [rows][q heads] tensor to fill, or None; workspace: a uint8 CUDA tensor of
    window_workspace bytes (one is allocated when None).  See
    kvpool_window_attend in include/kvpool.h."""
    import torch
    if not q.is_cuda:
        raise ValueError("window_attend: the tensors must be CUDA tensors")
    like = _like(q)
    index = like[2]
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return window_attend(q, k, v, q_len, k_start, k_len, window, n_sink, scale, out, lse, workspace, stream)
    raw = _stream_of(stream, index)
    rows = _rows(q, "q", like)
    if out is None:
        out, o = _fresh(q, stream, raw)
    else:
        o = _rows(out, "out", like, True)
    call = _window_call(q, like, rows, k, v, q_len, k_start, k_len, window, n_sink, scale, out, o, lse)
    L = lib()
    rc = L.kvpool_window_workspace(*call)
    if rc >= 0:
        nbytes = 0
        if workspace is not None:
            if workspace.get_device() != index or not workspace.is_contiguous():
                raise ValueError("window_attend: workspace must be a contiguous tensor on the queries' device")
            nbytes = workspace.numel() * workspace.element_size()
        elif rc > 0:
            nbytes = rc
            workspace = _fresh_bytes(rc, q.device, stream, raw)
        rc = L.kvpool_window_attend(*call, workspace.data_ptr() if nbytes else None, nbytes, raw)
    if rc != OK:
        raise KvpoolError(rc, "window_attend refused its arguments" if rc == ERR_INVALID_ARG else "window_attend: CUDA error")
    return out


def window_workspace(q, k, v, q_len, k_start, k_len, window: int, n_sink: int = 0, scale=None) -> int:
    """Workspace bytes of window_attend with these arguments."""
    import torch
    like = _like(q)
    with torch.cuda.device(like[2]):
        rows = _rows(q, "q", like)
        # an output like q, which may be a view that no output could have
        o = (rows[0], q.shape[1] * q.shape[2], q.shape[2], q.shape[1], 0)
        call = _window_call(q, like, rows, k, v, q_len, k_start, k_len, window, n_sink, scale, q, o, None)
        rc = int(lib().kvpool_window_workspace(*call))
    if rc < 0:
        raise KvpoolError(rc, "window_workspace refused its arguments")
    return rc


def window_check(stream=None) -> tuple:
    """(return code, device error flags) of the window_attend and Kv4Cache calls
    on the current device since the last check; synchronizes the stream."""
    w = C.c_uint32(0)
    rc = lib().kvpool_window_check(_stream(stream), C.byref(w))
    return int(rc), int(w.value)


def _window_call(q, like, q_rows, k, v, q_len, k_start, k_len, window, n_sink, scale, out, out_rows, lse):
    """(args, n, lengths) as kvpool_window_attend takes them (copies in bytes objects: quicker than array addresses)."""
    if k.shape != v.shape or out.shape != q.shape:
        raise ValueError("window_attend: k and v, and q and out, must have the same shape")
    z = 0
    if lse is not None:
        import torch
        z = _need(lse, "lse", torch.float32, q.shape[:2], like[2])
    ql, ks, kl = _i64(q_len), _i64(k_start), _i64(k_len)
    if not ql.size == ks.size == kl.size:
        raise ValueError("window_attend: q_len, k_start and k_len must have one value per segment")
    D = like[1]
    try:
        a = _WINDOW_ARGS.pack(_dtype(q), D, *q_rows, *_rows(k, "k", like), *_rows(v, "v", like), *out_rows, q.shape[0],
                              k.shape[0], z, window, n_sink, D ** -0.5 if scale is None else scale, 0)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"window_attend: {e}") from None
    return a, ql.size, ql.tobytes(), ks.tobytes(), kl.tobytes()


def kv4_page_bytes(kv_heads: int, head_dim: int, page_tokens: int) -> int:
    """Bytes of a page of a Kv4Cache."""
    n = int(lib().kvpool_kv4_page_bytes(kv_heads, head_dim, page_tokens))
    if n < 0:
        raise KvpoolError(n, "kv4_page_bytes: 1 to 1024 heads of 64 or 128, pages of 16 to 1024 tokens (a power of two)")
    return n


def _table(t, what: str, index: int) -> tuple:
    """(address, row stride, rows, ids per row) of a table of page ids."""
    import torch
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or t.dtype is not torch.int32 or t.get_device() != index or stride[1] != 1 and shape[1] > 1:
        raise ValueError(f"{what} must be a 2-D int32 tensor on cuda:{index} whose rows are contiguous")
    return t.data_ptr(), stride[0], shape[0], shape[1]


def _weights(w, what: str, n: int, heads: int, width: int, index: int) -> tuple:
    """(address, segment stride, head stride) of fp32 weights [segments][key heads][>= width]."""
    import torch
    shape, stride = w.shape, w.stride()
    if (len(shape) != 3 or w.dtype is not torch.float32 or w.get_device() != index or stride[2] != 1 and shape[2] > 1
            or shape[0] < n or shape[1] != heads or shape[2] < width):
        raise ValueError(f"{what} must be float32 [segments][key heads][at least {width} places] on cuda:{index}, places adjacent")
    return w.data_ptr(), stride[0], stride[1]


class Kv4Cache:
    """A paged cache of raw tokens held in 4 bits, in the caller's pages: a
    contiguous uint8 CUDA tensor [n_pages][kv4_page_bytes].  Segment i of a call
    is row i of the int32 CUDA table of page ids that the call is given; lengths
    and starts are host integers.  Nothing but the pages is kept between calls.
    See kvpool_kv4 in include/kvpool.h."""

    def __init__(self, pages, kv_heads: int, head_dim: int, page_tokens: int, k_scale: float = 1.0, v_scale: float = 1.0):
        import torch
        size = kv4_page_bytes(kv_heads, head_dim, page_tokens)
        if not pages.is_cuda or pages.dtype is not torch.uint8 or pages.dim() != 2 or pages.shape[1] != size or \
                not pages.is_contiguous() or pages.data_ptr() % 16:
            raise ValueError(f"Kv4Cache: pages must be a contiguous uint8 CUDA tensor [n_pages][{size}]")
        self.pages, self.kv_heads, self.head_dim, self.page_tokens = pages, kv_heads, head_dim, page_tokens
        self.k_scale, self.v_scale = k_scale, v_scale
        self.index, self.device = pages.get_device(), pages.device
        self._at = pages.data_ptr(), pages.shape[0]
        self._kind = kv_heads, head_dim, page_tokens, k_scale, v_scale, 0
        self._torch, self._lib = torch, lib()
        self._device_now, self._stream_now = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        self._types = {torch.bfloat16: BF16, torch.float32: F32}

    def _pack(self, table, n: int) -> bytes:
        ptr, stride, rows, width = _table(table, "table", self.index)
        if rows < n:
            raise ValueError("the table must have a row per segment")
        return _KV4.pack(*self._at, ptr, stride, rows, width, *self._kind)

    def _done(self, rc: int, what: str) -> None:
        if rc != OK:
            raise KvpoolError(rc, f"{what} refused its arguments" if rc == ERR_INVALID_ARG else f"{what}: CUDA error")

    def _two(self, start, length, what: str):
        a, b = _i64(start), _i64(length)
        if a.size != b.size:
            raise ValueError(f"{what}: one value of each kind per segment")
        return a, b

    def store(self, k, v, table, start, n_new, stream=None) -> None:
        """Store the next n_new[i] rows of k and v ([rows][key heads][dim],
        float32 or bfloat16) as the tokens of segment i from place start[i] on.
        See kvpool_kv4_store in include/kvpool.h."""
        if self._device_now() != self.index:
            with self._torch.cuda.device(self.index):
                return self.store(k, v, table, start, n_new, stream)
        start, n_new = self._two(start, n_new, "store")
        like = _like(k)
        if like[2] != self.index or like[1] != self.head_dim or k.shape != v.shape:
            raise ValueError("store: k and v must be CUDA tensors alike, of the cache's head dim and on its device")
        self._move(self._lib.kvpool_kv4_store, "store", like[0], k.shape[0], _rows(k, "k", like), _rows(v, "v", like), table,
                   start, n_new, stream)

    def load(self, table, start, length, dtype=None, out_k=None, out_v=None, stream=None) -> tuple:
        """(k, v): segment i's length[i] tokens from place start[i] on, as the
        values that they stand for (bfloat16 unless dtype or a given output says
        float32).  Where one output is given the other one is made like it.
        See kvpool_kv4_load in include/kvpool.h."""
        if self._device_now() != self.index:
            with self._torch.cuda.device(self.index):
                return self.load(table, start, length, dtype, out_k, out_v, stream)
        start, length = self._two(start, length, "load")
        if out_k is None and out_v is None:
            n, H, D = sum(length.tolist()), self.kv_heads, self.head_dim
            if dtype is None:
                dtype = self._torch.bfloat16
            out_k, out_v = self._empty((n, H, D), dtype, stream), self._empty((n, H, D), dtype, stream)
            k, v = (out_k.data_ptr(), H * D, D, H, 0), (out_v.data_ptr(), H * D, D, H, 0)
        else:
            if out_k is None or out_v is None:
                o = out_k if out_k is not None else out_v
                made = self._empty(o.shape, o.dtype if dtype is None else dtype, stream)
                out_k, out_v = (made, o) if out_k is None else (o, made)
            like = _like(out_k)
            if like[2] != self.index or like[1] != self.head_dim or out_k.shape != out_v.shape:
                raise ValueError("load: out_k and out_v must be CUDA tensors alike, of the cache's head dim and on its device")
            dtype, n, k, v = like[0], out_k.shape[0], _rows(out_k, "out_k", like, True), _rows(out_v, "out_v", like, True)
        self._move(self._lib.kvpool_kv4_load, "load", dtype, n, k, v, table, start, length, stream)
        return out_k, out_v

    def _empty(self, shape, dtype, stream):
        """A tensor whose memory belongs to the stream that will write it."""
        torch = self._torch
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        raw = _stream(stream)
        if raw == self._stream_now(self.index):
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(torch.cuda.ExternalStream(raw, device=self.device)):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def _move(self, call, what, dtype, n, k, v, table, start, length, stream) -> None:
        kind = self._types.get(dtype)
        if kind is None:
            raise ValueError("tensors must be float32 or bfloat16")
        rc = call(self._pack(table, start.size), kind, _HEADS.pack(*k), _HEADS.pack(*v), n, start.size, start.tobytes(),
                  length.tobytes(), self._stream_now(self.index) if stream is None else _stream(stream))
        if rc != OK:
            self._done(rc, what)

    def attend(self, q, table, q_len, k_len, scale=None, out=None, lse=None, weights=None, decay: float = 1.0, workspace=None,
               stream=None):
        """Attention of a ragged batch of queries, each segment's last ones, over
        its k_len[i] tokens; returns out ([rows][q heads][dim], like q, and q
        itself if given as out).  lse: a float32 [rows][q heads] tensor to fill, or
        None.  weights: None, or float32 accumulators [segments][key heads][places]
        that become decay times what they were plus the softmax weights that each
        token got from its head's queries.  workspace: a uint8 CUDA tensor of
        workspace() bytes (one is allocated when None).  No gradients flow through.
        See kvpool_kv4_attend in include/kvpool.h."""
        if self._device_now() != self.index:
            with self._torch.cuda.device(self.index):
                return self.attend(q, table, q_len, k_len, scale, out, lse, weights, decay, workspace, stream)
        if not q.is_cuda:
            raise ValueError("attend: q must be a CUDA tensor")
        raw = self._stream_now(self.index) if stream is None else _stream(stream)
        like = _like(q)
        rows = _rows(q, "q", like)
        if out is None:
            n, heads, dim = q.shape
            out = self._empty((n, heads, dim), like[0], stream)
            o = (out.data_ptr(), heads * dim if n > 1 else 0, dim if heads > 1 else 0, heads, 0)
        else:
            o = _rows(out, "out", like, True)
        call = self._call(q, like, rows, table, q_len, k_len, scale, out, o, lse, weights, decay)
        L = self._lib
        rc = L.kvpool_kv4_workspace(*call)
        if rc >= 0:
            nbytes = 0
            if workspace is not None:
                if workspace.get_device() != self.index or not workspace.is_contiguous():
                    raise ValueError("attend: workspace must be a contiguous tensor on the cache's device")
                nbytes = workspace.numel() * workspace.element_size()
            elif rc > 0:
                nbytes = rc
                workspace = self._empty((rc,), self._torch.uint8, stream)
            rc = L.kvpool_kv4_attend(*call, workspace.data_ptr() if nbytes else None, nbytes, raw)
        if rc != OK:
            self._done(rc, "attend")
        return out

    def workspace(self, q, table, q_len, k_len, scale=None, weights=None) -> int:
        """Workspace bytes of attend with these arguments."""
        import torch
        like = _like(q)
        with torch.cuda.device(self.index):
            rows = _rows(q, "q", like)
            # an output like q, which may be a view that no output could have
            o = (rows[0], q.shape[1] * q.shape[2], q.shape[2], q.shape[1], 0)
            rc = int(lib().kvpool_kv4_workspace(*self._call(q, like, rows, table, q_len, k_len, scale, q, o, None, weights, 1.0)))
        if rc < 0:
            raise KvpoolError(rc, "workspace refused its arguments")
        return rc

    def _call(self, q, like, q_rows, table, q_len, k_len, scale, out, out_rows, lse, weights, decay):
        shape, kind = q.shape, self._types.get(like[0])
        if kind is None:
            raise ValueError("tensors must be float32 or bfloat16")
        if like[1] != self.head_dim or like[2] != self.index or out.shape != shape:
            raise ValueError("attend: q and out must be alike, of the cache's head dim and on its device")
        ql, kl = self._two(q_len, k_len, "attend")
        z = 0 if lse is None else _need(lse, "lse", self._torch.float32, shape[:2], self.index)
        w = (0, 0, 0)
        if weights is not None:
            w = _weights(weights, "weights", ql.size, self.kv_heads, max(kl.tolist(), default=0), self.index)
        try:
            a = _KV4_ARGS.pack(kind, self.head_dim ** -0.5 if scale is None else scale, *q_rows, *out_rows, shape[0], z, *w, decay, 0)
        except (struct.error, OverflowError) as e:
            raise ValueError(f"attend: {e}") from None
        return self._pack(table, ql.size) + a, ql.size, ql.tobytes(), kl.tobytes()

    def evict(self, table, k_len, weights, keep: int, out_table, n_sink: int = 0, n_recent: int = 0, index=None,
              out_weights=None, stream=None) -> tuple:
        """Keep, of each segment's k_len[i] tokens and for every key head, the
        first n_sink, the last n_recent and the heaviest others, keep in all, in
        the pages of out_table (none of which is in table); returns (index,
        out_weights): the places they had ([segments][key heads][keep] int32, -1
        behind the last) and their weights (zeros behind).  See kvpool_kv4_evict in
        include/kvpool.h."""
        torch = self._torch
        if self._device_now() != self.index:
            with torch.cuda.device(self.index):
                return self.evict(table, k_len, weights, keep, out_table, n_sink, n_recent, index, out_weights, stream)
        kl = _i64(k_len)
        n, H = kl.size, self.kv_heads
        w = _weights(weights, "weights", n, H, max(kl.tolist(), default=0), self.index)
        ot = _table(out_table, "out_table", self.index)
        if index is None:
            index = self._empty((n, H, max(keep, 0)), torch.int32, stream)
            at = index.data_ptr()
        else:
            at = _need(index, "index", torch.int32, torch.Size((n, H, keep)), self.index)
        if out_weights is None:
            out_weights = self._empty((n, H, max(keep, 0)), torch.float32, stream)
            ow, width = (out_weights.data_ptr(), H * keep, keep), keep
        else:
            ow, width = _weights(out_weights, "out_weights", n, H, keep, self.index), out_weights.shape[2]
        try:
            a = _KV4_EVICT.pack(*ot, *w, *ow, at, width, keep, n_sink, n_recent)
        except (struct.error, OverflowError) as e:
            raise ValueError(f"evict: {e}") from None
        rc = self._lib.kvpool_kv4_evict(self._pack(table, n) + a, n, kl.tobytes(),
                                        self._stream_now(self.index) if stream is None else _stream(stream))
        if rc != OK:
            self._done(rc, "evict")
        return index, out_weights


class Pool:
    """A two-pool KV cache living in a caller-owned device arena."""

    def __init__(self, cfg: PoolConfig, arena=None, stream=None):
        self.L = lib()
        self.cfg = cfg
        self._c = cfg.to_c()
        self.arena = arena
        h = C.c_void_p()
        if cfg.flags & FLAG_NO_DEVICE:
            rc = self.L.kvpool_create(C.byref(self._c), None, 0, None, C.byref(h))
        else:
            nbytes = arena.numel() * arena.element_size()
            rc = self.L.kvpool_create(C.byref(self._c), arena.data_ptr(), nbytes, _stream(stream), C.byref(h))
        if rc != OK:
            raise KvpoolError(rc, "kvpool_create refused the configuration")
        self.h = h
        self.n_layers = len(cfg.layer_kinds)
        self.HD = cfg.heads * cfg.head_dim
        self.XD = cfg.idx_heads * cfg.idx_dim

    def __del__(self):
        if getattr(self, "h", None):
            self.L.kvpool_destroy(self.h)
            self.h = None

    def last_error(self) -> str:
        return self.L.kvpool_last_error(self.h).decode()

    def _check(self, rc: int, what: str) -> int:
        if rc != OK:
            raise KvpoolError(rc, f"{what}: {self.last_error()}")
        return rc

    # ---- lifecycle ----
    def alloc_request(self) -> int:
        r = C.c_int32()
        self._check(self.L.kvpool_alloc_request(self.h, C.byref(r)), "alloc_request")
        return r.value

    def free_request(self, req: int) -> None:
        self._check(self.L.kvpool_free_request(self.h, req), "free_request")

    def share_prefix(self, dst, src, n_tokens, win_k, win_v, stream=None, check=True) -> int:
        rc = self.L.kvpool_share_prefix(self.h, dst, src, n_tokens, _ptr(win_k), _ptr(win_v), _stream(stream))
        return self._check(rc, "share_prefix") if check else rc

    # ---- prefix images (sealed blocks in page-locked host memory) ----
    def fingerprint(self) -> int:
        return int(self.L.kvpool_fingerprint(self.h))

    def image_bytes(self, n_tokens: int, flags: int = 0) -> int:
        return int(self.L.kvpool_image_bytes(self.h, n_tokens, flags))

    def export_prefix(self, req, n_tokens, flags=0, out=None, stream=None, check=True):
        """Write the image of req's first n_tokens tokens into `out` (a
        page-locked uint8 host tensor; allocated when None) and return it.  The
        copy runs in stream order: the image is complete once the stream has
        reached it."""
        if out is None:
            import torch
            out = torch.empty(max(self.image_bytes(n_tokens, flags), 64), dtype=torch.uint8, pin_memory=True)
        addr, nbytes = _host_buffer(out)
        rc = self.L.kvpool_export_prefix(self.h, req, n_tokens, flags, addr, nbytes, _stream(stream))
        if check:
            self._check(rc, "export_prefix")
            return out
        return rc

    def import_prefix(self, dst, image, win_k=None, win_v=None, stream=None, check=True) -> int:
        """Restore an image (page-locked host memory) into the fresh request
        dst; win_k / win_v: the recomputed window for an image without one."""
        addr, nbytes = _host_buffer(image)
        rc = self.L.kvpool_import_prefix(self.h, dst, addr, nbytes, _ptr(win_k), _ptr(win_v), _stream(stream))
        return self._check(rc, "import_prefix") if check else rc

    # ---- HiSparse: inactive CSA entries off the GPU ----
    def host_slot_bytes(self) -> int:
        return int(self.L.kvpool_host_slot_bytes(self.h))

    def set_host_pool(self, pool=None, check=True):
        """Give the pool its host slots (a page-locked uint8 host tensor; one is
        allocated when None) and return it; the caller keeps it alive."""
        if pool is None:
            import torch
            pool = torch.empty(max(self.cfg.csa_host_slots * self.host_slot_bytes(), 16), dtype=torch.uint8,
                               pin_memory=True)
        addr, nbytes = _host_buffer(pool)
        rc = self.L.kvpool_set_host_pool(self.h, addr, nbytes)
        if check:
            self._check(rc, "set_host_pool")
            self._host_pool = pool
            return pool
        return rc

    def offload(self, block_ids, stream=None, check=True) -> int:
        ids = _i32(block_ids)
        rc = self.L.kvpool_offload(self.h, ids.size, ids.ctypes.data, _stream(stream))
        return self._check(rc, "offload") if check else rc

    def fetch(self, block_ids, stream=None, check=True) -> int:
        ids = _i32(block_ids)
        rc = self.L.kvpool_fetch(self.h, ids.size, ids.ctypes.data, _stream(stream))
        return self._check(rc, "fetch") if check else rc

    def block_location(self, block_id: int):
        """(rc, loc): loc >= 0 a GPU slot, < 0 host slot -1 - loc."""
        loc = C.c_int32()
        rc = self.L.kvpool_block_location(self.h, block_id, C.byref(loc))
        return rc, loc.value

    def epoch(self) -> int:
        return int(self.L.kvpool_epoch(self.h))

    def block_activity(self, block_ids, stream=None) -> np.ndarray:
        ids = _i32(block_ids)
        out = np.zeros(max(ids.size, 1), np.uint32)
        rc = self.L.kvpool_block_activity(self.h, ids.size, ids.ctypes.data,
                                          out.ctypes.data, _stream(stream))
        self._check(rc, "block_activity")
        return out[:ids.size]

    def inactive_blocks(self, idle: int, cap: int = 1 << 20, stream=None) -> np.ndarray:
        ids = np.zeros(max(cap, 1), np.int32)
        n = self.L.kvpool_inactive_blocks(self.h, idle, ids.ctypes.data, cap, _stream(stream))
        if n < 0:
            self._check(n, "inactive_blocks")
        return ids[:min(n, cap)].copy()

    def append(self, req_ids, n_new, k, v, idx_k, stream=None, check=True) -> int:
        req, nn = _i32(req_ids), _i32(n_new)
        rc = self.L.kvpool_append(self.h, req.size, req.ctypes.data, nn.ctypes.data,
                                  _ptr(k), _ptr(v), _ptr(idx_k), _stream(stream))
        return self._check(rc, "append") if check else rc

    def decode_attend(self, layer, req_ids, q, q_idx, top_k, out, topk_out=None, stream=None, check=True) -> int:
        req = _i32(req_ids)
        rc = self.L.kvpool_decode_attend(self.h, layer, req.size, req.ctypes.data, _ptr(q),
                                         _ptr(q_idx), top_k, _ptr(out), _ptr(topk_out), _stream(stream))
        return self._check(rc, "decode_attend") if check else rc

    def decode_attend_shared(self, layer, req_ids, n_shared, q, q_idx, top_k, out, topk_out=None, stream=None,
                             check=True) -> int:
        """decode_attend of requests whose first n_shared tokens are the same
        blocks, whose HCA entries are read once for all of them where that is
        the quicker way (set_share_bytes)."""
        req = _i32(req_ids)
        rc = self.L.kvpool_decode_attend_shared(self.h, layer, req.size, req.tobytes(), n_shared, _ptr(q), _ptr(q_idx),
                                                top_k, _ptr(out), _ptr(topk_out), _stream(stream))
        return self._check(rc, "decode_attend_shared") if check else rc

    def set_share_bytes(self, nbytes: int) -> None:
        """The reading that decode_attend_shared has to save to share entries (negative: the measured rule)."""
        self._check(self.L.kvpool_set_share_bytes(self.h, nbytes), "set_share_bytes")

    # ---- queries ----
    def request_info(self, req: int, cap: int = 1 << 16):
        info = _Info()
        ids = np.zeros(max(cap, 1), np.int32)
        rc = self.L.kvpool_request_info(self.h, req, C.byref(info), ids.ctypes.data, cap)
        if rc != OK:
            return rc, None, None
        d = {f: getattr(info, f) for f, _ in _Info._fields_}
        return rc, d, ids[:info.n_blocks].copy()

    def block_refcount(self, b: int) -> int:
        return self.L.kvpool_block_refcount(self.h, b)

    def free_block_count(self) -> int:
        return self.L.kvpool_free_block_count(self.h)

    def layout(self, layer: Optional[int] = None):
        lo = _Layout()
        ll = _LayerLayout()
        rc = self.L.kvpool_get_layout(self.h, C.byref(lo), -1 if layer is None else layer,
                                      None if layer is None else C.byref(ll))
        self._check(rc, "get_layout")
        d = {f: getattr(lo, f) for f, _ in _Layout._fields_}
        if layer is not None:
            d.update({f: getattr(ll, f) for f, _ in _LayerLayout._fields_})
        return d

    def wait_selftest(self, stream=None) -> None:
        """A kernel whose barrier wait runs out (see kvpool_wait_selftest)."""
        self._check(self.L.kvpool_wait_selftest(self.h, _stream(stream)), "wait_selftest")

    def check_device(self, stream=None) -> int:
        w = C.c_uint32()
        rc = self.L.kvpool_check_device(self.h, _stream(stream), C.byref(w))
        if rc != OK:
            raise KvpoolError(rc, f"check_device: {self.last_error()} (flags {w.value:#x})")
        return w.value

    def profile_enable(self, on: bool = True, kinds=None, count: bool = False) -> None:
        """Record the launches of the given kernel kinds (indexes into
        KERNEL_NAMES; all kinds when None), or stop recording.  count: every
        launch of every kind also adds its kernel count and algorithmic bytes
        to the totals, with no events (kinds=[] counts without timing)."""
        mask = 0
        if on:
            mask = (1 << len(KERNEL_NAMES)) - 1 if kinds is None else sum(1 << int(k) for k in set(kinds))
            if count:
                mask |= PROFILE_COUNT
        self._check(self.L.kvpool_profile_enable(self.h, mask), "profile_enable")

    def profile_timeline(self, cap: int = 4096):
        """[(kernel name, start ms, end ms)] of the recorded launches."""
        buf = np.zeros((cap, 3), np.float32)
        n = self.L.kvpool_profile_timeline(self.h, cap, buf.ctypes.data)
        if n < 0:
            raise KvpoolError(n, "profile_timeline")
        return [(KERNEL_NAMES[int(k)], float(a), float(b)) for k, a, b in buf[:n]]

    def profile_read(self, kernel: int):
        ms, n, b = C.c_double(), C.c_int64(), C.c_int64()
        self._check(self.L.kvpool_profile_read(self.h, kernel, C.byref(ms), C.byref(n), C.byref(b)), "profile_read")
        return ms.value, n.value, b.value
