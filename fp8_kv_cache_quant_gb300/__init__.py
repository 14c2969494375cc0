"""Python binding of libfp8kv.so (FP8 KV-cache quantisation and FP8 attention, sm_103a).

Argument marshalling only: every step of the computation runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors (used for device memory and streams); the
C entry points receive their raw pointers.  The binding has the C ABI's names:
``kv_quant_cache``, ``fp8_decode_attn``, ``fp8_prefill_attn`` and the size queries; the rotary
cache writes ``kv_rope_cache`` and ``kv_block_cache``; ``fp8_block_decode_attn`` and
``fp8_block_prefill_attn`` over block-scaled pools.

The library must have been built (``python -m fp8_kv_cache_quant_gb300.build`` or
``__graft_entry__.build()``); importing the binding does not load it, calling an
entry point without it raises ``RuntimeError``.  There is no fallback path.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp8kv.so")

OK, INVALID_ARG, UNSUPPORTED, CUDA_ERROR = 0, 1, 2, 3
SCALE_PER_TENSOR, SCALE_PER_HEAD = 0, 1
KV_E4M3, KV_E5M2 = 0, 1
FAULT_BLOCK_ID, FAULT_SLOT, FAULT_CONTEXT, FAULT_TIMEOUT, FAULT_QLEN, FAULT_WORKSPACE = 1, 2, 4, 8, 16, 32
FAULT_POSITION = 64

# Entry points declared by include/fp8kv.h (checked by the tests).
EXPORTS = (
    "fkv_status_string", "fkv_version", "kv_quant_cache", "fp8_decode_attn_workspace_size",
    "fp8_decode_attn_num_splits", "fp8_decode_attn", "fkv_prefill_block_n", "fp8_prefill_attn",
    "fp8_decode_attn_noalloc", "fp8_decode_attn_split_blocks", "fkv_decode_block_n", "kv_quant_cache_clips",
    "fp8_decode_step", "fkv_set_decode_wait_limit_ns", "kv_rope_cache", "kv_block_cache",
    "fp8_block_decode_attn", "fp8_block_prefill_attn",
)
NOALLOC_WORKSPACE_BYTES = 16 << 20


class FkvError(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn}: {text} (status {status})")
        self.status = status


class _LayerCache(ctypes.Structure):
    _fields_ = [("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("num_blocks", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("kv_format", ctypes.c_int32)]


class _BlockCache(ctypes.Structure):
    _fields_ = [("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _Rope(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("max_positions", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


_lib = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libfp8kv.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libfp8kv.so not built ({p}); run __graft_entry__.build()")
    lib = ctypes.CDLL(p)
    c_i32, c_vp, c_f, c_sz = ctypes.c_int32, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
    lib.fkv_status_string.restype = ctypes.c_char_p
    lib.fkv_status_string.argtypes = [ctypes.c_int]
    lib.fkv_version.restype = c_i32
    lib.fkv_set_decode_wait_limit_ns.restype = None
    lib.fkv_set_decode_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
    lib.kv_quant_cache.restype = ctypes.c_int
    lib.kv_quant_cache.argtypes = [c_vp, c_vp, c_vp, c_i32, _LayerCache, c_vp, c_vp, ctypes.c_int, c_i32, c_vp,
                                   c_i32, c_vp, c_vp]
    lib.kv_quant_cache_clips.restype = ctypes.c_int
    lib.kv_quant_cache_clips.argtypes = [c_vp, c_vp, c_vp, c_i32, _LayerCache, c_vp, c_vp, ctypes.c_int, c_i32, c_vp,
                                         c_i32, c_vp, c_vp, c_vp]
    lib.fp8_decode_attn_workspace_size.restype = c_sz
    lib.fp8_decode_attn_workspace_size.argtypes = [c_i32] * 7
    lib.fp8_decode_attn_num_splits.restype = c_i32
    lib.fp8_decode_attn_num_splits.argtypes = [c_i32] * 7
    lib.fp8_decode_attn_split_blocks.restype = c_i32
    lib.fp8_decode_attn_split_blocks.argtypes = [c_i32] * 7
    lib.fkv_decode_block_n.restype = c_i32
    lib.fkv_decode_block_n.argtypes = [c_i32, c_i32]
    lib.fp8_decode_attn.restype = ctypes.c_int
    lib.fp8_decode_attn.argtypes = [c_vp, c_i32, c_i32, _LayerCache, c_vp, c_i32, c_vp, c_vp, c_vp, c_vp,
                                    ctypes.c_int, c_f, c_i32, c_i32, c_vp, c_i32, c_vp, c_vp, c_sz, c_i32, c_vp,
                                    c_vp]
    lib.fp8_decode_step.restype = ctypes.c_int
    lib.fp8_decode_step.argtypes = [c_vp, c_vp] + lib.fp8_decode_attn.argtypes
    lib.fp8_decode_attn_noalloc.restype = ctypes.c_int
    lib.fp8_decode_attn_noalloc.argtypes = [c_vp, c_i32, c_i32, _LayerCache, c_vp, c_i32, c_vp, c_vp, c_vp, c_vp,
                                            ctypes.c_int, c_f, c_i32, c_i32, c_vp, c_i32, c_vp, c_i32, c_vp, c_vp]
    lib.fkv_prefill_block_n.restype = c_i32
    lib.fkv_prefill_block_n.argtypes = [c_i32]
    lib.fp8_prefill_attn.restype = ctypes.c_int
    lib.fp8_prefill_attn.argtypes = [c_vp, c_vp, c_i32, c_i32, c_i32, _LayerCache, c_vp, c_i32, c_vp, c_vp, c_vp,
                                     c_vp, ctypes.c_int, c_f, c_i32, c_i32, c_i32, c_i32, c_vp, c_i32, c_vp, c_vp,
                                     c_vp]
    c_i64 = ctypes.c_int64
    lib.kv_rope_cache.restype = ctypes.c_int
    lib.kv_rope_cache.argtypes = [c_vp, c_i64, c_vp, c_i64, c_i32, c_vp, c_i64, c_vp, c_i64, c_vp, c_vp, c_i32, _Rope,
                                  _LayerCache, c_vp, c_vp, ctypes.c_int, c_i32, c_vp, c_i32, c_vp, c_vp]
    lib.kv_block_cache.restype = ctypes.c_int
    lib.kv_block_cache.argtypes = [c_vp, c_i64, c_vp, c_i64, c_i32, c_vp, c_i64, c_vp, c_i64, c_i32, c_vp, c_i32, c_i32,
                                   _Rope, _BlockCache, c_vp, c_i32, c_vp, c_vp, c_vp]
    lib.fp8_block_decode_attn.restype = ctypes.c_int
    lib.fp8_block_decode_attn.argtypes = [c_vp, c_i32, c_i32, _BlockCache, c_vp, c_i32, c_vp, c_f, c_i32, c_vp, c_vp,
                                          c_sz, c_i32, c_vp, c_vp]
    lib.fp8_block_prefill_attn.restype = ctypes.c_int
    lib.fp8_block_prefill_attn.argtypes = [c_vp, c_vp, c_i32, c_i32, c_i32, c_i32, _BlockCache, c_vp, c_i32, c_vp, c_f,
                                           c_i32, c_i32, c_vp, c_vp, c_vp]
    if path is None:
        _lib = lib
    return lib


def _check(fn: str, st: int):
    if st != OK:
        raise FkvError(fn, st, load_library().fkv_status_string(st).decode())


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


@dataclasses.dataclass
class LayerCache:
    """One layer's K/V pools: uint8 (FP8 codes of ``kv_format``: KV_E4M3 or KV_E5M2) or
    bfloat16 tensors [num_blocks][Hkv][16][D]."""

    k_cache: torch.Tensor
    v_cache: torch.Tensor
    kv_format: int = 0

    @property
    def num_blocks(self):
        return self.k_cache.shape[0]

    @property
    def num_kv_heads(self):
        return self.k_cache.shape[1]

    @property
    def block_size(self):
        return self.k_cache.shape[2]

    @property
    def head_dim(self):
        return self.k_cache.shape[3]

    def c(self) -> _LayerCache:
        return _LayerCache(self.k_cache.data_ptr(), self.v_cache.data_ptr(), self.num_blocks, self.block_size,
                           self.num_kv_heads, self.head_dim, self.kv_format)

    @staticmethod
    def empty(num_blocks, num_kv_heads, head_dim, bf16=False, device="cuda", block_size=16, kv_format=0):
        dt = torch.bfloat16 if bf16 else torch.uint8
        shape = (num_blocks, num_kv_heads, block_size, head_dim)
        return LayerCache(torch.empty(shape, dtype=dt, device=device), torch.empty(shape, dtype=dt, device=device),
                          kv_format)


def _mask_arg(skip_layer_mask):
    if skip_layer_mask is None:
        return None, 0, None
    arr = np.ascontiguousarray(np.asarray(skip_layer_mask, dtype=np.uint8))
    return arr.ctypes.data, int(arr.size), arr   # keep arr alive in the caller


def kv_quant_cache(k, v, slot_mapping, cache: LayerCache, k_scale=None, v_scale=None, gran=SCALE_PER_TENSOR,
                   layer=0, skip_layer_mask=None, fault=None, stream=None):
    lib = load_library()
    mp, nl, keep = _mask_arg(skip_layer_mask)
    st = lib.kv_quant_cache(_ptr(k), _ptr(v), _ptr(slot_mapping), int(k.shape[0]), cache.c(), _ptr(k_scale),
                            _ptr(v_scale), int(gran), int(layer), mp, nl, _ptr(fault), _stream(stream))
    del keep
    _check("kv_quant_cache", st)


def kv_quant_cache_clips(k, v, slot_mapping, cache: LayerCache, k_scale, v_scale, gran=SCALE_PER_TENSOR,
                         clip_counts=None, layer=0, skip_layer_mask=None, fault=None, stream=None):
    """kv_quant_cache that also adds the numbers of clipped K and V elements to
    ``clip_counts`` (device int64 [2], created zeroed when None); returns it."""
    lib = load_library()
    if clip_counts is None:
        clip_counts = torch.zeros(2, dtype=torch.int64, device=k.device)
    mp, nl, keep = _mask_arg(skip_layer_mask)
    st = lib.kv_quant_cache_clips(_ptr(k), _ptr(v), _ptr(slot_mapping), int(k.shape[0]), cache.c(), _ptr(k_scale),
                                  _ptr(v_scale), int(gran), int(layer), mp, nl, _ptr(clip_counts), _ptr(fault),
                                  _stream(stream))
    del keep
    _check("kv_quant_cache_clips", st)
    return clip_counts


def fp8_decode_attn_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, max_blocks, window=0,
                                   num_splits=0) -> int:
    return int(load_library().fp8_decode_attn_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                              max_blocks, window, num_splits))


def fp8_decode_attn_num_splits(batch, num_q_heads, num_kv_heads, head_dim, max_blocks, window=0,
                               num_splits=0) -> int:
    return int(load_library().fp8_decode_attn_num_splits(batch, num_q_heads, num_kv_heads, head_dim, max_blocks,
                                                          window, num_splits))


def fp8_decode_attn_split_blocks(batch, num_q_heads, num_kv_heads, head_dim, max_blocks, window=0,
                                 num_splits=0) -> int:
    return int(load_library().fp8_decode_attn_split_blocks(batch, num_q_heads, num_kv_heads, head_dim, max_blocks,
                                                            window, num_splits))


def fkv_decode_block_n(head_dim: int, bf16_layer: bool = False, kv_format: int = 0) -> int:
    kind = 1 if bf16_layer else (2 if kv_format == KV_E5M2 else 0)
    return int(load_library().fkv_decode_block_n(head_dim, kind))


def decode_workspace(batch, num_q_heads, cache: LayerCache, max_blocks, window=0, num_splits=0, device="cuda"):
    """A zero-filled decode workspace (the split counters at its start must be zero when a
    call begins; every call leaves them zero)."""
    n = fp8_decode_attn_workspace_size(batch, num_q_heads, cache.num_kv_heads, cache.head_dim, max_blocks,
                                       window, num_splits)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def fp8_decode_attn(q, cache: LayerCache, block_table, context_lens, q_scale=None, k_scale=None, v_scale=None,
                    gran=SCALE_PER_TENSOR, softmax_scale=0.0, window=0, layer=0, skip_layer_mask=None, out=None,
                    workspace=None, num_splits=0, fault=None, stream=None):
    lib = load_library()
    B, Hq, D = q.shape
    max_blocks = int(block_table.shape[1])
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=q.device)
    if workspace is None:
        workspace = decode_workspace(B, Hq, cache, max_blocks, window, num_splits, q.device)
    mp, nl, keep = _mask_arg(skip_layer_mask)
    st = lib.fp8_decode_attn(_ptr(q), B, Hq, cache.c(), _ptr(block_table), max_blocks, _ptr(context_lens),
                             _ptr(q_scale), _ptr(k_scale), _ptr(v_scale), int(gran), float(softmax_scale),
                             int(window), int(layer), mp, nl, _ptr(out), _ptr(workspace),
                             int(workspace.numel() * workspace.element_size()), int(num_splits), _ptr(fault),
                             _stream(stream))
    del keep
    _check("fp8_decode_attn", st)
    return out


def fp8_decode_step(k_new, v_new, q, cache: LayerCache, block_table, context_lens, q_scale=None, k_scale=None,
                    v_scale=None, gran=SCALE_PER_TENSOR, softmax_scale=0.0, window=0, layer=0, skip_layer_mask=None,
                    out=None, workspace=None, num_splits=0, fault=None, stream=None):
    """kv_quant_cache of the current token (k_new, v_new: bf16 [batch][num_kv_heads][head_dim], written at
    position context_lens[b] - 1) and fp8_decode_attn in one launch (e4m3 layers)."""
    lib = load_library()
    B, Hq, D = q.shape
    max_blocks = int(block_table.shape[1])
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=q.device)
    if workspace is None:
        workspace = decode_workspace(B, Hq, cache, max_blocks, window, num_splits, q.device)
    mp, nl, keep = _mask_arg(skip_layer_mask)
    st = lib.fp8_decode_step(_ptr(k_new), _ptr(v_new), _ptr(q), B, Hq, cache.c(), _ptr(block_table), max_blocks,
                             _ptr(context_lens), _ptr(q_scale), _ptr(k_scale), _ptr(v_scale), int(gran),
                             float(softmax_scale), int(window), int(layer), mp, nl, _ptr(out), _ptr(workspace),
                             int(workspace.numel() * workspace.element_size()), int(num_splits), _ptr(fault),
                             _stream(stream))
    del keep
    _check("fp8_decode_step", st)
    return out


def fp8_decode_attn_noalloc(q, cache: LayerCache, block_table, context_lens, q_scale=None, k_scale=None,
                            v_scale=None, gran=SCALE_PER_TENSOR, softmax_scale=0.0, window=0, layer=0,
                            skip_layer_mask=None, out=None, num_splits=0, fault=None, stream=None):
    """fp8_decode_attn without a workspace: the library's fixed device scratch is used
    (see include/fp8kv.h for its size limit and the sharing rule)."""
    lib = load_library()
    B, Hq, D = q.shape
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=q.device)
    mp, nl, keep = _mask_arg(skip_layer_mask)
    st = lib.fp8_decode_attn_noalloc(_ptr(q), B, Hq, cache.c(), _ptr(block_table), int(block_table.shape[1]),
                                     _ptr(context_lens), _ptr(q_scale), _ptr(k_scale), _ptr(v_scale), int(gran),
                                     float(softmax_scale), int(window), int(layer), mp, nl, _ptr(out),
                                     int(num_splits), _ptr(fault), _stream(stream))
    del keep
    _check("fp8_decode_attn_noalloc", st)
    return out


def fkv_prefill_block_n(head_dim: int) -> int:
    return int(load_library().fkv_prefill_block_n(head_dim))


def fp8_prefill_attn(q, cu_seqlens_q, max_q_len, cache: LayerCache, block_table, context_lens, q_scale=None,
                     k_scale=None, v_scale=None, gran=SCALE_PER_TENSOR, softmax_scale=0.0, causal=True, window=0,
                     promote_every=1, layer=0, skip_layer_mask=None, out=None, fault=None, stream=None):
    lib = load_library()
    N, Hq, D = q.shape
    B = int(cu_seqlens_q.shape[0]) - 1
    if out is None:
        out = torch.empty((N, Hq, D), dtype=torch.bfloat16, device=q.device)
    mp, nl, keep = _mask_arg(skip_layer_mask)
    st = lib.fp8_prefill_attn(_ptr(q), _ptr(cu_seqlens_q), B, Hq, int(max_q_len), cache.c(), _ptr(block_table),
                              int(block_table.shape[1]), _ptr(context_lens), _ptr(q_scale), _ptr(k_scale),
                              _ptr(v_scale), int(gran), float(softmax_scale), int(bool(causal)), int(window),
                              int(promote_every), int(layer), mp, nl, _ptr(out), _ptr(fault), _stream(stream))
    del keep
    _check("fp8_prefill_attn", st)
    return out


# ------------------------------------------------------------------ rotary cache writes, block-scaled cache

@dataclasses.dataclass
class Rope:
    """A rotary position embedding: ``cos_sin`` float32 [max_positions][rot_dim], row p holding
    rot_dim / 2 cosines, then rot_dim / 2 sines; ``interleaved`` pairs neighbours (2 i, 2 i + 1)
    instead of the halves (i, i + rot_dim / 2)."""

    cos_sin: torch.Tensor
    interleaved: bool = False

    def c(self) -> _Rope:
        t = self.cos_sin
        return _Rope(t.data_ptr(), t.shape[0], t.shape[1], int(self.interleaved))

    @staticmethod
    def table(max_positions, rot_dim, base=10000.0, device="cuda"):
        """The table of angles p * base^(-2 i / rot_dim), evaluated in float64."""
        inv = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
        a = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * inv
        return torch.cat((a.cos(), a.sin()), 1).float()


@dataclasses.dataclass
class BlockCache:
    """One layer's block-scaled pools: e4m3 codes (uint8) [num_blocks][Hkv][16][D] and the
    float32 scales [num_blocks][Hkv] of every block and KV head, for K and for V."""

    k_cache: torch.Tensor
    v_cache: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    @staticmethod
    def empty(num_blocks, num_kv_heads, head_dim, device="cuda", block_size=16):
        shape = (num_blocks, num_kv_heads, block_size, head_dim)
        return BlockCache(*(torch.empty(shape, dtype=torch.uint8, device=device) for _ in range(2)),
                          *(torch.empty(shape[:2], dtype=torch.float32, device=device) for _ in range(2)))


# The checks below run before every launch, and a small call's time is host time: what passes costs a
# few attribute reads, and messages are built only for what does not.

def _refuse(fn, what):
    raise ValueError(f"{fn}: {what}")


def _check_tensors(fn, device, *wanted):
    """Each (name, tensor or None, dtype, shape): contiguous, of that type and shape, on `device`."""
    for name, t, dtype, shape in wanted:
        if t is not None and not (t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device):
            _refuse(fn, f"{name} is {t.dtype} {tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}; "
                        f"wanted {dtype} {tuple(shape)} on {device}, contiguous")


def _rows(fn, device, name, t, n, heads, d):
    """The token stride of a bf16 tensor [n][heads][d] whose rows are consecutive (a slice of a wider
    projection's output serves)."""
    if not (t.dtype is torch.bfloat16 and t.shape == (n, heads, d) and t.device == device):
        _refuse(fn, f"{name} is {t.dtype} {tuple(t.shape)} on {t.device}; wanted torch.bfloat16 {(n, heads, d)} on {device}")
    if n == 0:
        return heads * d
    s = t.stride()
    if s[2] != 1 or (heads > 1 and s[1] != d):
        _refuse(fn, f"{name}'s rows of {heads} x {d} elements are not consecutive (strides {s})")
    return s[0] if n > 1 else heads * d


def _launch(fn, device, stream, *args):
    """The library's fn(*args, stream) with the tensors' device current; stream None: that device's current
    stream."""
    call = getattr(_lib or load_library(), fn)
    index = device.index
    s = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream)
    if index == torch._C._cuda_getDevice():
        st = call(*args, s)
    else:
        with torch.cuda.device(device):
            st = call(*args, s)
    if st != OK:
        _check(fn, st)


def _device(fn, t):
    """The CUDA device of t, whose number of dimensions is 3."""
    if not t.is_cuda or t.dim() != 3:
        _refuse(fn, f"a tensor of shape {tuple(t.shape)} on {t.device}; wanted [n][heads][head_dim] on a CUDA device")
    return t.device


def _query_rows(fn, device, q, q_out, n, d):
    """(q, its stride, q_out, its stride, heads) as the entry points take them, and the output tensor, of
    an optional query tensor [n][Hq][d]."""
    if q is None:
        if q_out is not None:
            _refuse(fn, "q_out without q")
        return (None, 0, None, 0, 0), None
    hq = q.shape[1] if q.dim() == 3 else -1
    stride = _rows(fn, device, "q", q, n, hq, d)
    if q_out is None:
        q_out = torch.empty((n, hq, d), dtype=torch.bfloat16, device=device)
    return (q.data_ptr(), stride, q_out.data_ptr(), _rows(fn, device, "q_out", q_out, n, hq, d), hq), q_out


def kv_rope_cache(q, k, v, positions, slot_mapping, rope: Rope, cache: LayerCache, k_scale=None, v_scale=None,
                  gran=SCALE_PER_TENSOR, layer=0, skip_layer_mask=None, q_out=None, fault=None, stream=None):
    """kv_quant_cache of K turned for its positions and of V, and the turned queries (bf16, returned; rows of
    skipped tokens are not written).  q, k, v: bf16 [n][heads][D], rows may be slices of a wider tensor; q may
    be None, q_out may be q.  positions, slot_mapping: int64 [n]."""
    fn = "kv_rope_cache"
    device = _device(fn, k)
    n, h, d = k.shape
    ks, vs = _rows(fn, device, "k", k, n, h, d), _rows(fn, device, "v", v, n, h, d)
    qa, q_out = _query_rows(fn, device, q, q_out, n, d)
    mp, nl, keep = _mask_arg(skip_layer_mask)
    pool_t = torch.bfloat16 if keep is not None and 0 <= layer < nl and keep[layer] else torch.uint8
    pool = (cache.k_cache.shape[0], h, cache.k_cache.shape[2] if cache.k_cache.dim() == 4 else 16, d)
    scales = (h if gran == SCALE_PER_HEAD else 1,)
    cs = rope.cos_sin
    _check_tensors(fn, device, ("positions", positions, torch.int64, (n,)), ("slot_mapping", slot_mapping, torch.int64, (n,)),
                   ("k_cache", cache.k_cache, pool_t, pool), ("v_cache", cache.v_cache, pool_t, pool),
                   ("k_scale", k_scale, torch.float32, scales), ("v_scale", v_scale, torch.float32, scales),
                   ("cos_sin", cs, torch.float32, cs.shape if cs.dim() == 2 else (0, 0)), ("fault", fault, torch.int32, (1,)))
    _launch(fn, device, stream, *qa, k.data_ptr(), ks, v.data_ptr(), vs, positions.data_ptr(), slot_mapping.data_ptr(), n,
            rope.c(), _LayerCache(cache.k_cache.data_ptr(), cache.v_cache.data_ptr(), pool[0], pool[2], h, d, cache.kv_format),
            _ptr(k_scale), _ptr(v_scale), gran, layer, mp, nl, _ptr(fault))
    del keep
    return q_out


def _block_cache(fn, device, cache, h, d):
    """The C structure of a block-scaled cache of h KV heads and head_dim d."""
    k = cache.k_cache
    nb, bs = (k.shape[0], k.shape[2]) if k.dim() == 4 else (0, 16)
    pool, scales = (nb, h, bs, d), (nb, h)
    _check_tensors(fn, device, ("k_cache", k, torch.uint8, pool), ("v_cache", cache.v_cache, torch.uint8, pool),
                   ("k_scale", cache.k_scale, torch.float32, scales), ("v_scale", cache.v_scale, torch.float32, scales))
    return _BlockCache(k.data_ptr(), cache.v_cache.data_ptr(), cache.k_scale.data_ptr(), cache.v_scale.data_ptr(), nb, bs, h, d)


def kv_block_cache(k, v, cu_seqlens, max_q_len, cache: BlockCache, block_table, context_lens, rope: Optional[Rope] = None,
                   q=None, q_out=None, fault=None, stream=None):
    """Append each sequence's new tokens (rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of k, v and q, the last of
    its context_lens[b] tokens) to a block-scaled cache, K and q turned for their positions when ``rope`` is
    given; returns the turned queries (None without q)."""
    fn = "kv_block_cache"
    device = _device(fn, k)
    n, h, d = k.shape
    ks, vs = _rows(fn, device, "k", k, n, h, d), _rows(fn, device, "v", v, n, h, d)
    qa, q_out = _query_rows(fn, device, q, q_out, n, d)
    b, mb = block_table.shape if block_table.dim() == 2 else (-1, 0)
    cs = None if rope is None else rope.cos_sin
    _check_tensors(fn, device, ("cu_seqlens", cu_seqlens, torch.int32, (b + 1,)), ("block_table", block_table, torch.int32, (b, mb)),
                   ("context_lens", context_lens, torch.int32, (b,)), ("fault", fault, torch.int32, (1,)),
                   ("cos_sin", cs, torch.float32, cs.shape if cs is not None and cs.dim() == 2 else (0, 0)))
    c = _block_cache(fn, device, cache, h, d)
    _launch(fn, device, stream, *qa, k.data_ptr(), ks, v.data_ptr(), vs, n, cu_seqlens.data_ptr(), b, max_q_len,
            _Rope() if rope is None else rope.c(), c, block_table.data_ptr(), mb, context_lens.data_ptr(), _ptr(fault))
    return q_out


def _attn_args(fn, q, rows, cache, block_table, context_lens, out, fault):
    device = _device(fn, q)
    n, hq, d = q.shape
    k = cache.k_cache
    b, mb = block_table.shape if block_table.dim() == 2 else (-1, 0)
    want = (n if rows is None else b, hq, d)
    if out is None:
        out = torch.empty(want, dtype=torch.bfloat16, device=device)
    _check_tensors(fn, device, ("q", q, torch.bfloat16, want), ("out", out, torch.bfloat16, want),
                   ("block_table", block_table, torch.int32, (b, mb)), ("context_lens", context_lens, torch.int32, (b,)),
                   ("fault", fault, torch.int32, (1,)))
    return device, out, _block_cache(fn, device, cache, k.shape[1] if k.dim() == 4 else 0, d), n, hq, b, mb


def fp8_block_decode_attn(q, cache: BlockCache, block_table, context_lens, softmax_scale=0.0, window=0, out=None,
                          workspace=None, num_splits=0, fault=None, stream=None):
    """One decode step over a block-scaled cache: q bf16 [batch][Hq][D] (not rounded further), out bf16.  The
    workspace is fp8_decode_attn's (``decode_workspace`` makes one; zero-filled before its first call)."""
    fn = "fp8_block_decode_attn"
    device, out, c, _, hq, b, mb = _attn_args(fn, q, "batch", cache, block_table, context_lens, out, fault)
    if workspace is None:
        n = fp8_decode_attn_workspace_size(b, hq, c.num_kv_heads, c.head_dim, mb, window, num_splits)
        workspace = torch.zeros(max(n, 256), dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous():
        _refuse(fn, f"workspace on {workspace.device}; wanted contiguous on {device}")
    _launch(fn, device, stream, q.data_ptr(), b, hq, c, block_table.data_ptr(), mb, context_lens.data_ptr(), softmax_scale,
            window, out.data_ptr(), workspace.data_ptr(), workspace.nbytes, num_splits, _ptr(fault))
    return out


def fp8_block_prefill_attn(q, cu_seqlens_q, max_q_len, cache: BlockCache, block_table, context_lens, softmax_scale=0.0,
                           causal=True, window=0, out=None, fault=None, stream=None):
    """Ragged chunks of queries (rows cu_seqlens_q[b] .. of q bf16 [total][Hq][D]) over a block-scaled cache."""
    fn = "fp8_block_prefill_attn"
    device, out, c, n, hq, b, mb = _attn_args(fn, q, None, cache, block_table, context_lens, out, fault)
    _check_tensors(fn, device, ("cu_seqlens_q", cu_seqlens_q, torch.int32, (b + 1,)))
    _launch(fn, device, stream, q.data_ptr(), cu_seqlens_q.data_ptr(), n, b, hq, max_q_len, c, block_table.data_ptr(), mb,
            context_lens.data_ptr(), softmax_scale, bool(causal), window, out.data_ptr(), _ptr(fault))
    return out
