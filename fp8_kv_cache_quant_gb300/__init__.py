"""Python binding of libfp8kv.so (FP8 KV-cache quantisation and FP8 attention, sm_103a).

Argument marshalling only (part of it compiled, csrc/binding.cpp): every step of the
computation runs in the library's CUDA kernels.  Tensors are torch CUDA tensors (used for device memory and streams); the
C entry points receive their raw pointers.  The binding has the C ABI's names:
``kv_quant_cache``, ``fp8_decode_attn``, ``fp8_prefill_attn`` and the size queries; the rotary
cache writes ``kv_rope_cache`` and ``kv_block_cache`` (positions of one axis or several);
``fp8_block_decode_attn``, ``fp8_block_shared_decode_attn`` (sequences that share their first
tokens) and ``fp8_block_prefill_attn`` over block-scaled pools; ``fp8_block_attn_weights``, what
cached keys receive of the attention, and ``kv_block_evict``, which keeps the heaviest.

The library must have been built (``python -m fp8_kv_cache_quant_gb300.build`` or
``__graft_entry__.build()``); importing the binding does not load it, calling an
entry point without it raises ``RuntimeError``.  There is no fallback path.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional, Sequence

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
    "kv_rope_cache_axes", "kv_block_cache_axes", "kv_block_evict",
    "fp8_block_shared_decode_attn_workspace_size", "fp8_block_shared_decode_attn",
    "fp8_block_attn_weights_workspace_size", "fp8_block_attn_weights",
    "fp8_block_decode_attn_workspace_size", "fp8_block_decode_attn", "fp8_block_prefill_attn",
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


class _Axes(ctypes.Structure):
    _fields_ = [("positions", ctypes.c_void_p), ("axis_stride", ctypes.c_int64), ("num_axes", ctypes.c_int32),
                ("pair_axis", ctypes.c_void_p)]


class _Rope(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("max_positions", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


_lib = None
_compiled = None


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
    lib.kv_rope_cache_axes.restype = ctypes.c_int
    lib.kv_rope_cache_axes.argtypes = [_Axes if i == 9 else t for i, t in enumerate(lib.kv_rope_cache.argtypes)]
    lib.kv_block_cache_axes.restype = ctypes.c_int
    lib.kv_block_cache_axes.argtypes = lib.kv_block_cache.argtypes[:10] + [_Axes] + lib.kv_block_cache.argtypes[10:]
    lib.fp8_block_decode_attn.restype = ctypes.c_int
    lib.fp8_block_decode_attn.argtypes = [c_vp, c_i32, c_i32, _BlockCache, c_vp, c_i32, c_vp, c_f, c_i32, c_vp, c_vp,
                                          c_sz, c_vp, c_vp]
    lib.fp8_block_decode_attn_workspace_size.restype = c_sz
    lib.fp8_block_decode_attn_workspace_size.argtypes = [c_i32] * 4
    lib.fp8_block_prefill_attn.restype = ctypes.c_int
    lib.fp8_block_prefill_attn.argtypes = [c_vp, c_vp, c_i32, c_i32, c_i32, c_i32, _BlockCache, c_vp, c_i32, c_vp, c_f,
                                           c_i32, c_i32, c_vp, c_vp, c_vp]
    lib.kv_block_evict.restype = ctypes.c_int
    lib.kv_block_evict.argtypes = [_BlockCache, c_vp, c_i32, c_i32, c_vp, c_vp, c_i32, c_i32, c_i32, c_i32, c_vp, c_i32, c_vp, c_vp,
                                   c_vp, c_i32, c_vp, c_vp]
    lib.fp8_block_shared_decode_attn_workspace_size.restype = c_sz
    lib.fp8_block_shared_decode_attn_workspace_size.argtypes = [c_i32] * 5
    lib.fp8_block_shared_decode_attn.restype = ctypes.c_int
    lib.fp8_block_shared_decode_attn.argtypes = [c_vp, c_i32, c_i32, _BlockCache, c_vp, c_i32, c_vp, c_vp, c_vp, c_i32, c_f, c_i32, c_vp,
                                                 c_vp, c_sz, c_vp, c_vp]
    lib.fp8_block_attn_weights_workspace_size.restype = c_sz
    lib.fp8_block_attn_weights_workspace_size.argtypes = [c_i32] * 7
    lib.fp8_block_attn_weights.restype = ctypes.c_int
    lib.fp8_block_attn_weights.argtypes = [c_vp, c_vp, c_i32, c_i32, c_i32, c_i32, _BlockCache, c_vp, c_i32, c_vp, c_f, c_f, c_vp,
                                           c_i32, c_vp, c_sz, c_vp, c_vp]
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

class _PairAxes:
    """Rope.axes: checked when assigned, and kept as the calls take them besides."""

    def __get__(self, rope, cls=None):
        return None if rope is None else rope._axes

    def __set__(self, rope, axes):
        if axes is None:
            if rope._axes is not None:
                del rope._axes, rope.pair_axis, rope.pair_args      # (the class has those of no axes)
            return
        x, n = np.asarray(axes), rope.cos_sin.shape[1]
        if x.ndim != 1 or 2 * x.size != n or x.dtype.kind not in "iu" or x.min() < 0 or x.max() > 3:
            raise ValueError(f"Rope: axes names an axis from 0 to 3 for each of the {n // 2} pairs")
        rope._axes = tuple(x.tolist())      # (changed by assigning others)
        rope.pair_axis = np.ascontiguousarray(x, np.uint8)
        rope.pair_args = (rope.pair_axis.ctypes.data, rope.pair_axis.size)


@dataclasses.dataclass
class Rope:
    """A rotary position embedding: ``cos_sin`` float32 [max_positions][rot_dim], row p holding
    rot_dim / 2 cosines, then rot_dim / 2 sines; ``interleaved`` pairs neighbours (2 i, 2 i + 1)
    instead of the halves (i, i + rot_dim / 2).  ``axes``: for positions of several axes (time, height, width),
    the axis, 0 to 3, of each of the rot_dim / 2 pairs; positions are then int64 [axes][n].
    pair_axis holds them as bytes, pair_args these bytes' address and number."""

    cos_sin: torch.Tensor
    interleaved: bool = False
    axes: Optional[Sequence[int]] = _PairAxes()

    _axes = pair_axis = None
    pair_args = (None, 0)

    # A copy, also in another process, has bytes and an address of its own.
    def __getstate__(self):
        own = ("_axes", "pair_axis", "pair_args")
        return {**{k: v for k, v in self.__dict__.items() if k not in own}, "axes": self.axes}

    def __setstate__(self, state):
        for k, v in state.items():
            setattr(self, k, v)

    @staticmethod
    def sections(*pairs):
        """``axes`` of consecutive sections: pairs[0] pairs of axis 0, then pairs[1] of axis 1, ..."""
        return [a for a, n in enumerate(pairs) for _ in range(n)]

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


def load_binding():
    """The compiled part of this binding (built for this Python and this torch): the checks and calls of the functions
    below, whose small calls are bound by the host."""
    global _compiled
    if _compiled is None:
        import importlib.util

        from .build import binding_path
        load_library()
        path = binding_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} not built; run __graft_entry__.build()")
        spec = importlib.util.spec_from_file_location(__name__ + "._binding", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _compiled = module
    return _compiled


def _current(stream, index):
    """A context in which the raw stream of device `index` is the current one."""
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=index) if stream else torch.cuda.default_stream(index))


def _allocating(fn, on, stream):
    """A context in which the device of the tensor `on` and the stream (None: that device's current one) are current."""
    index = on.get_device()
    if index < 0:
        raise ValueError(f"{fn}: the tensors are not on a CUDA device")
    return torch.cuda.device(index) if stream is None else _current(_stream(stream), index)


def _call(fn, on, stream, *args):
    """fn of the compiled binding, with the device of the tensor `on` and the stream current (what the call
    allocates belongs to that stream); stream None: that device's current stream.  Returns its tensor."""
    index = on.get_device()
    if index < 0:
        raise ValueError(f"{fn}: the tensors are not on a CUDA device")
    call = getattr(_compiled or load_binding(), fn)
    current = torch._C._cuda_getCurrentRawStream(index)
    s = current if stream is None else _stream(stream)
    if s == current and index == torch._C._cuda_getDevice():
        st, out = call(s, *args)
    else:
        with _current(s, index):
            st, out = call(s, *args)
    if st != OK:
        _check(fn, st)
    return out


def kv_rope_cache(q, k, v, positions, slot_mapping, rope: Rope, cache: LayerCache, k_scale=None, v_scale=None,
                  gran=SCALE_PER_TENSOR, layer=0, skip_layer_mask=None, q_out=None, fault=None, stream=None):
    """kv_quant_cache of K turned for its positions and of V, and the turned queries (bf16, returned; rows of
    skipped tokens are not written).  q, k, v: bf16 [n][heads][D], rows may be slices of a wider tensor; q may
    be None, q_out may be q.  positions, slot_mapping: int64 [n]; with ``rope.axes`` positions is int64 [axes][n]."""
    mp, nl, keep = _mask_arg(skip_layer_mask)
    skipped = keep is not None and 0 <= layer < nl and bool(keep[layer])
    several = rope.pair_axis is not None
    return _call("kv_rope_cache_axes" if several else "kv_rope_cache", k, stream, q, k, v, positions, slot_mapping, rope.cos_sin,
                 rope.interleaved, *(rope.pair_args if several else ()), cache.k_cache, cache.v_cache, cache.kv_format, k_scale,
                 v_scale, gran, layer, mp, nl, skipped, q_out, fault)


def kv_block_cache(k, v, cu_seqlens, max_q_len, cache: BlockCache, block_table, context_lens, rope: Optional[Rope] = None,
                   q=None, q_out=None, fault=None, stream=None, positions=None):
    """Append each sequence's new tokens (rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of k, v and q, the last of
    its context_lens[b] tokens) to a block-scaled cache, K and q turned for their positions when ``rope`` is
    given; returns the turned queries (None without q).  ``positions``: int64 [n], or [axes][n] with ``rope.axes``,
    what the rows are turned for (None: their places in the cache)."""
    given = ()
    if positions is not None:
        given = (*((None, 0) if rope is None else rope.pair_args), positions)
    elif rope is not None and rope.pair_axis is not None:
        raise ValueError("kv_block_cache: a rope of several axes takes positions")
    return _call("kv_block_cache_axes" if given else "kv_block_cache", k, stream, k, v, cu_seqlens, max_q_len, cache.k_cache,
                 cache.v_cache, cache.k_scale, cache.v_scale, block_table, context_lens, None if rope is None else rope.cos_sin,
                 rope is not None and rope.interleaved, *given, q, q_out, fault)


def fp8_block_decode_attn_workspace_size(batch, num_q_heads, num_kv_heads, head_dim) -> int:
    return int(load_library().fp8_block_decode_attn_workspace_size(batch, num_q_heads, num_kv_heads, head_dim))


def block_decode_workspace(batch, num_q_heads, cache: BlockCache, stream=None):
    """A workspace of fp8_block_decode_attn, zero-filled on the stream (calls that may overlap on the GPU each
    need one)."""
    _, h, _, d = cache.k_cache.shape
    with _allocating("fp8_block_decode_attn", cache.k_cache, stream):
        n = fp8_block_decode_attn_workspace_size(batch, num_q_heads, h, d)
        return torch.zeros(max(n, 256), dtype=torch.uint8, device=cache.k_cache.device)


def fp8_block_decode_attn(q, cache: BlockCache, block_table, context_lens, softmax_scale=0.0, window=0, out=None,
                          workspace=None, fault=None, stream=None):
    """One decode step over a block-scaled cache: q bf16 [batch][Hq][D] (not rounded further), out bf16.
    ``workspace``: of block_decode_workspace (when None, one is made and cleared for the call: a loop keeps its own)."""
    if workspace is None:
        workspace = block_decode_workspace(q.shape[0], q.shape[1], cache, stream)
    return _call("fp8_block_decode_attn", q, stream, q, cache.k_cache, cache.v_cache, cache.k_scale, cache.v_scale, block_table,
                 context_lens, softmax_scale, window, out, workspace, fault)


def fp8_block_prefill_attn(q, cu_seqlens_q, max_q_len, cache: BlockCache, block_table, context_lens, softmax_scale=0.0,
                           causal=True, window=0, out=None, fault=None, stream=None):
    """Ragged chunks of queries (rows cu_seqlens_q[b] .. of q bf16 [total][Hq][D]) over a block-scaled cache."""
    return _call("fp8_block_prefill_attn", q, stream, q, cu_seqlens_q, max_q_len, cache.k_cache, cache.v_cache, cache.k_scale,
                 cache.v_scale, block_table, context_lens, softmax_scale, causal, window, out, fault)


# ------------------------------------------------------------------ long and shared contexts

def fp8_block_shared_decode_attn_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, num_groups) -> int:
    return int(load_library().fp8_block_shared_decode_attn_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, num_groups))


def block_shared_workspace(batch, num_q_heads, cache: BlockCache, num_groups, stream=None):
    """A workspace of fp8_block_shared_decode_attn, zero-filled on the stream (calls that may overlap on the GPU each
    need one)."""
    _, h, _, d = cache.k_cache.shape
    with _allocating("fp8_block_shared_decode_attn", cache.k_cache, stream):
        n = fp8_block_shared_decode_attn_workspace_size(batch, num_q_heads, h, d, num_groups)
        return torch.zeros(max(n, 256), dtype=torch.uint8, device=cache.k_cache.device)


def fp8_block_shared_decode_attn(q, cache: BlockCache, block_table, context_lens, group_starts, shared_lens, softmax_scale=0.0,
                                 window=0, out=None, workspace=None, fault=None, stream=None):
    """fp8_block_decode_attn of a batch whose group i, sequences group_starts[i] .. group_starts[i + 1] - 1 (int32 [groups + 1]), has its
    first shared_lens[i] tokens (int32 [groups]) in common: their keys and values are read and multiplied once per group.
    ``workspace``: of block_shared_workspace (when None, one is made and cleared for the call: a loop keeps its own)."""
    if workspace is None:
        workspace = block_shared_workspace(q.shape[0], q.shape[1], cache, shared_lens.shape[0], stream)
    return _call("fp8_block_shared_decode_attn", q, stream, q, cache.k_cache, cache.v_cache, cache.k_scale, cache.v_scale, block_table,
                 context_lens, group_starts, shared_lens, softmax_scale, window, out, workspace, fault)


def fp8_block_attn_weights_workspace_size(batch, total_q, max_q_len, num_q_heads, num_kv_heads, head_dim, max_blocks) -> int:
    return int(load_library().fp8_block_attn_weights_workspace_size(batch, total_q, max_q_len, num_q_heads, num_kv_heads,
                                                                    head_dim, max_blocks))


def attn_weights_workspace(batch, total_q, max_q_len, num_q_heads, cache: BlockCache, max_blocks, stream=None):
    """A workspace of fp8_block_attn_weights (calls that may overlap on the GPU each need one).  For few queries (at most 16 rows of
    a KV head and sequence) it grows with the table's width, ``max_blocks``: see include/fp8kv.h."""
    _, h, _, d = cache.k_cache.shape
    with _allocating("fp8_block_attn_weights", cache.k_cache, stream):
        n = fp8_block_attn_weights_workspace_size(batch, total_q, max_q_len, num_q_heads, h, d, max_blocks)
        return torch.empty(max(n, 256), dtype=torch.uint8, device=cache.k_cache.device)


def fp8_block_attn_weights(q, cu_seqlens_q, max_q_len, cache: BlockCache, block_table, context_lens, weights, softmax_scale=0.0,
                           decay=1.0, workspace=None, fault=None, stream=None):
    """Add to ``weights`` (float32 [batch][Hkv][>= T]) the softmax weight that each key of a block-scaled cache receives from
    the chunk's queries (the last tokens of their sequences; rows cu_seqlens_q[b] .. of q bf16 [total][Hq][D]), summed over the
    queries and a group's heads: decay * before + new for older keys (decay 0: what was there is not read), new for the
    chunk's own.  ``workspace``: of attn_weights_workspace (None: made for the call).  Returns weights."""
    if workspace is None:
        workspace = attn_weights_workspace(block_table.shape[0], q.shape[0], max_q_len, q.shape[1], cache, block_table.shape[1], stream)
    return _call("fp8_block_attn_weights", q, stream, q, cu_seqlens_q, max_q_len, cache.k_cache, cache.v_cache, cache.k_scale,
                 cache.v_scale, block_table, context_lens, weights, softmax_scale, decay, workspace, fault)


def kv_block_evict(cache: BlockCache, block_table, context_lens, weights, budget, new_table, sink=0, recent=0, new_weights=None,
                   new_lens=None, kept=None, fault=None, stream=None):
    """Cut every sequence to min(T, budget) tokens per KV head: the first ``sink``, the last ``recent`` and, of the others,
    those with the largest ``weights`` (float32 [batch][Hkv][>= T], equal ones by index), copied in order to the blocks
    of ``new_table`` (none of them read by the call).  Returns (new_lens int32 [batch], kept int32 [batch][Hkv][budget]:
    the kept tokens' old indices, then -1); their weights go to ``new_weights`` when given."""
    dev = cache.k_cache.device
    if new_lens is None or kept is None:
        with _allocating("kv_block_evict", cache.k_cache, stream):
            if new_lens is None:
                new_lens = torch.empty(block_table.shape[0], dtype=torch.int32, device=dev)
            if kept is None:
                kept = torch.empty(block_table.shape[0], cache.k_cache.shape[1], max(budget, 0), dtype=torch.int32, device=dev)
    _call("kv_block_evict", cache.k_cache, stream, cache.k_cache, cache.v_cache, cache.k_scale, cache.v_scale, block_table,
          context_lens, weights, budget, sink, recent, new_table, new_weights, new_lens, kept, fault)
    return new_lens, kept
