"""Thin ctypes binding of libdflash2.so (declared in include/dflash2.h).

Argument marshalling only: each function checks shapes and dtypes of torch
CUDA tensors, passes their data pointers and the current CUDA stream to the
C entry point of the same name, and raises :class:`Dflash2Error` on a
non-OK status.  Every step of the hot path runs in the library's kernels;
there is no fallback.  If the shared library is missing the first call
raises: build it with ``python -c "import __graft_entry__ as g; g.build()"``.

PyTorch provides device memory and streams only.  Workspaces are caller-owned
device buffers; the helpers here allocate them with torch when not given.  A call
with ``stream`` allocates what it was not given (workspace, outputs, error word) in
that stream; that its inputs are ready there is the caller's to see to.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import NamedTuple

import numpy as np
import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdflash2.so")
_lock = threading.Lock()
_lib = None

OK = 0
F32, BF16 = 0, 1
KV_NATIVE, KV_E4M3 = 0, 1
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3
GATE_ACTS = {"none": 0, "sigmoid": 1, "tanh": 2}
DEVERR_ID_RANGE = 0x1
DEVERR_TIMEOUT = 0x2
DEVERR_SHORT = 0x4
DEVINFO_TOPK_FALLBACK = 0x100
ABI_VERSION = 9

# Every symbol include/dflash2.h declares.
EXPORTS = (
    "dflash2_status_string", "dflash2_abi_version", "dflash2_grouped_conv",
    "dflash2_unary_topk_workspace_size", "dflash2_unary_topk_workspace_min",
    "dflash2_unary_topk", "dflash2_selector_walk_workspace_size", "dflash2_selector_walk",
    "dflash2_d2t_remap", "dflash2_selector_walk_noalloc", "dflash2_philox_uniforms",
    "dflash2_conv_prepare", "dflash2_conv_finish", "dflash2_verify_workspace_size",
    "dflash2_verify", "dflash2_selector_project", "dflash2_selector_walk_projected",
    "dflash2_unary_topk_launches", "dflash2_topk_merge", "dflash2_quantize_rows_e4m3",
    "dflash2_unary_topk_fp8_workspace_size", "dflash2_unary_topk_fp8",
    "dflash2_quantize_rows_nvfp4", "dflash2_unary_topk_nvfp4_workspace_size",
    "dflash2_unary_topk_nvfp4", "dflash2_nvfp4_scale_tiles_size", "dflash2_nvfp4_tile_scales",
    "dflash2_kv_cache_write", "dflash2_kv_cache_read", "dflash2_tree_attention_workspace_size",
    "dflash2_tree_attention", "dflash2_prompt_attention_workspace_size",
    "dflash2_prompt_attention", "dflash2_quantize_blocks_e4m3",
    "dflash2_linear_fp8_blocks_workspace_size", "dflash2_linear_fp8_blocks",
    "dflash2_sublayer_norm", "dflash2_sublayer_join", "dflash2_rotary", "dflash2_rotary_kv_write",
)
NOALLOC_SCRATCH_BYTES = 4 << 20


class Dflash2Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = library().dflash2_status_string(status).decode()
        super().__init__(f"{fn}: {msg} (status {status})")


def library():
    """Load libdflash2.so once and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: the CUDA extension is not built "
                "(run `python -c \"import __graft_entry__ as g; g.build()\"`)")
        lib = ctypes.CDLL(_LIB_PATH)
        P, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                ctypes.c_float, ctypes.c_size_t)
        lib.dflash2_status_string.argtypes = [i32]
        lib.dflash2_status_string.restype = ctypes.c_char_p
        lib.dflash2_abi_version.argtypes = []
        lib.dflash2_abi_version.restype = i32
        lib.dflash2_grouped_conv.argtypes = [P, P, P, i64, P, i64, i32, i32, i32, i32, i32, P]
        lib.dflash2_grouped_conv.restype = i32
        lib.dflash2_unary_topk_workspace_size.argtypes = [i64, i64, i32, i32]
        lib.dflash2_unary_topk_workspace_size.restype = sz
        lib.dflash2_unary_topk_workspace_min.argtypes = [i64, i64, i32, i32]
        lib.dflash2_unary_topk_workspace_min.restype = sz
        lib.dflash2_unary_topk.argtypes = [P, P, i64, i32, i64, i64, f32, f32, i32, i32, P, P, P,
                                           sz, P, P]
        lib.dflash2_unary_topk.restype = i32
        lib.dflash2_selector_walk_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.dflash2_selector_walk_workspace_size.restype = sz
        lib.dflash2_selector_walk.argtypes = [P, P, P, P, i64, P, P, P, P, P, P, i32, i32, i32,
                                              i32, i32, i32, P, P, P, P, sz, P, P]
        lib.dflash2_selector_walk.restype = i32
        lib.dflash2_d2t_remap.argtypes = [P, P, i64, i64, i64, P, P, P]
        lib.dflash2_d2t_remap.restype = i32
        lib.dflash2_selector_walk_noalloc.argtypes = [P, P, P, P, i64, P, P, P, P, P, P, i32, i32,
                                                      i32, i32, i32, i32, P, P, P, P, P]
        lib.dflash2_selector_walk_noalloc.restype = i32
        lib.dflash2_philox_uniforms.argtypes = [ctypes.c_uint64, ctypes.c_uint64, P, i64, P, P]
        lib.dflash2_philox_uniforms.restype = i32
        lib.dflash2_conv_prepare.argtypes = [P, P, P, i64, i32, i32, i32, i32, i32, P, P, P, P]
        lib.dflash2_conv_prepare.restype = i32
        lib.dflash2_conv_finish.argtypes = [P, P, P, i64, i32, i32, i32, i32, i32, P, P]
        lib.dflash2_conv_finish.restype = i32
        lib.dflash2_verify_workspace_size.argtypes = [i32, i32, i64]
        lib.dflash2_verify_workspace_size.restype = sz
        lib.dflash2_verify.argtypes = [P, i64, P, P, P, P, P, P, i32, i32, i32, i32, P, P, P, sz,
                                       P, P]
        lib.dflash2_verify.restype = i32
        lib.dflash2_selector_project.argtypes = [P, P, i32, i32, i32, i32, i32, i32, P, sz, P, P]
        lib.dflash2_selector_project.restype = i32
        lib.dflash2_selector_walk_projected.argtypes = [P, P, i64, P, P, P, P, P, P, i32, i32, i32,
                                                        i32, i32, i32, P, P, P, P, sz, P, P]
        lib.dflash2_selector_walk_projected.restype = i32
        lib.dflash2_quantize_rows_e4m3.argtypes = [P, i64, i32, i32, P, P, P]
        lib.dflash2_quantize_rows_e4m3.restype = i32
        lib.dflash2_unary_topk_fp8_workspace_size.argtypes = [i64, i32, i64, i32]
        lib.dflash2_unary_topk_fp8_workspace_size.restype = sz
        lib.dflash2_unary_topk_fp8.argtypes = [P, i32, P, P, i64, i32, i64, i64, f32, f32, i32, P,
                                               P, P, sz, P, P]
        lib.dflash2_unary_topk_fp8.restype = i32
        lib.dflash2_quantize_rows_nvfp4.argtypes = [P, i64, i32, i32, P, P, P, P]
        lib.dflash2_quantize_rows_nvfp4.restype = i32
        lib.dflash2_unary_topk_nvfp4_workspace_size.argtypes = [i64, i32, i64, i32]
        lib.dflash2_unary_topk_nvfp4_workspace_size.restype = sz
        lib.dflash2_unary_topk_nvfp4.argtypes = [P, i32, P, P, f32, i64, i32, i64, i64, f32, f32,
                                                 i32, P, P, P, sz, P, P]
        lib.dflash2_unary_topk_nvfp4.restype = i32
        lib.dflash2_nvfp4_scale_tiles_size.argtypes = [i64, i32]
        lib.dflash2_nvfp4_scale_tiles_size.restype = sz
        lib.dflash2_nvfp4_tile_scales.argtypes = [P, i64, i32, P, P]
        lib.dflash2_nvfp4_tile_scales.restype = i32
        lib.dflash2_topk_merge.argtypes = [P, P, P, i32, i64, i32, i32, P, P, P, P]
        lib.dflash2_topk_merge.restype = i32
        lib.dflash2_kv_cache_write.argtypes = [P, P, i64, i64, P, i64, i32, i32, i32, i64, i32,
                                               i32, P, P, P, P, P, P]
        lib.dflash2_kv_cache_write.restype = i32
        lib.dflash2_kv_cache_read.argtypes = [P, P, P, P, P, i64, i32, i32, i32, i64, i32, i32, P,
                                              P, P, P]
        lib.dflash2_kv_cache_read.restype = i32
        lib.dflash2_tree_attention_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        lib.dflash2_tree_attention_workspace_size.restype = sz
        lib.dflash2_tree_attention.argtypes = [P, i64, P, P, P, P, P, i32, i64, i32, P, P, P, i32,
                                               i32, i32, i32, i32, i32, f32, i32, i32, P, P, P, sz,
                                               P, P]
        lib.dflash2_tree_attention.restype = i32
        lib.dflash2_prompt_attention_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        lib.dflash2_prompt_attention_workspace_size.restype = sz
        lib.dflash2_prompt_attention.argtypes = [P, P, P, i64, i64, i64, P, i32, i32, i32, i32,
                                                 i32, f32, i32, P, P, P, sz, P, P]
        lib.dflash2_prompt_attention.restype = i32
        lib.dflash2_quantize_blocks_e4m3.argtypes = [P, i64, i64, i32, i32, P, P, P]
        lib.dflash2_quantize_blocks_e4m3.restype = i32
        lib.dflash2_linear_fp8_blocks_workspace_size.argtypes = [i64, i32, i32]
        lib.dflash2_linear_fp8_blocks_workspace_size.restype = sz
        lib.dflash2_linear_fp8_blocks.argtypes = [P, i64, i32, P, P, P, P, i64, i32, i32, i32, P, P,
                                                  sz, P, P]
        lib.dflash2_linear_fp8_blocks.restype = i32
        lib.dflash2_sublayer_norm.argtypes = [P, i64, i32, P, f32, f32, i64, i32, i32, P, P, P]
        lib.dflash2_sublayer_norm.restype = i32
        lib.dflash2_sublayer_join.argtypes = [P, i64, i32, P, i64, P, P, i32, i64, i32, f32, P, f32,
                                              f32, i64, i32, i32, P, i64, P, P, P]
        lib.dflash2_sublayer_join.restype = i32
        lib.dflash2_rotary.argtypes = [P, i64, P, i64, P, i32, P, P, i32, i32, f32, i64, i32, i32,
                                       i32, i32, P, i64, P, i64, P, P]
        lib.dflash2_rotary.restype = i32
        lib.dflash2_rotary_kv_write.argtypes = [P, i64, P, i64, P, i64, P, i32, P, P, i32, i32, f32,
                                                P, i64, i32, i32, i32, i32, i64, i32, i32, P, i64,
                                                P, i64, P, P, P, P, P, P]
        lib.dflash2_rotary_kv_write.restype = i32
        lib.dflash2_unary_topk_launches.argtypes = [i64, i64, i32, f32, i32]
        lib.dflash2_unary_topk_launches.restype = i32
        if lib.dflash2_abi_version() != ABI_VERSION:
            raise RuntimeError("libdflash2.so ABI version mismatch; rebuild it")
        _lib = lib
        return lib


def _check(fn: str, status: int):
    if status != OK:
        raise Dflash2Error(fn, status)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t.dtype}: fp32 or bf16 only")


def _ptr(t):  # the argument types make a void * of it
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:  # torch.cuda.current_stream() without building a Stream object
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _need(t: torch.Tensor, name: str, dtype=None, shape=None):
    if (t.is_cuda and t.is_contiguous() and (dtype is None or t.dtype == dtype)
            and (shape is None or t.shape == shape)):
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _empty(shape, dtype, device, stream):
    """A tensor that belongs to the stream the call runs on: when it is dropped, its memory goes
    to later work of that stream, not to the current one's while the call still uses it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _workspace(size: int, device, stream):
    return _empty(max(1, size), torch.uint8, device, stream)


def _error_word(device, stream):
    """A device error word, cleared in the call's own stream."""
    if stream is None:
        return torch.zeros(1, dtype=torch.int32, device=device)
    with torch.cuda.stream(stream):
        return torch.zeros(1, dtype=torch.int32, device=device)


# ---- entry points -----------------------------------------------------------------

def grouped_conv(x, base, delta, block_size: int, group_size: int, taps: int, out=None,
                 delta_row_stride: int | None = None, stream=None):
    """dflash2_grouped_conv: x [n, hidden], base [taps, hidden], delta rows of
    [taps, hidden/group_size] (row stride delta_row_stride elements)."""
    n, hidden = x.shape
    for t, nm in ((x, "x"), (base, "base"), (delta, "delta")):
        _need(t, nm, x.dtype)
    if out is None:
        out = _empty(x.shape, x.dtype, x.device, stream)
    _need(out, "out", x.dtype, x.shape)
    groups = hidden // group_size
    if delta_row_stride is None:
        delta_row_stride = taps * groups
    if delta.numel() < (n - 1) * delta_row_stride + taps * groups if n else False:
        raise ValueError("delta is too small for n rows at this row stride")
    _check("dflash2_grouped_conv", library().dflash2_grouped_conv(
        _ptr(x), _ptr(base), _ptr(delta), delta_row_stride, _ptr(out), n, hidden, group_size,
        taps, block_size, _dtype_code(x), _stream(stream)))
    return out


def unary_topk_workspace_size(rows: int, draft_vocab: int, top_k: int, dtype_code: int) -> int:
    return int(library().dflash2_unary_topk_workspace_size(rows, draft_vocab, top_k, dtype_code))


def unary_topk_workspace_min(rows: int, draft_vocab: int, top_k: int, dtype_code: int) -> int:
    return int(library().dflash2_unary_topk_workspace_min(rows, draft_vocab, top_k, dtype_code))


def unary_topk(h, lm_head, target_vocab: int, mult: float, cap: float, top_k: int,
               cand_ids=None, cand_u=None, workspace=None, err=None, stream=None):
    """dflash2_unary_topk: top_k (ids, u) per row of h against lm_head."""
    rows, hidden = h.shape
    draft_vocab = lm_head.shape[0]
    _need(h, "h")
    _need(lm_head, "lm_head", h.dtype)
    code = _dtype_code(h)
    dev = h.device
    if cand_ids is None:
        cand_ids = _empty((rows, top_k), torch.int64, dev, stream)
    if cand_u is None:
        cand_u = _empty((rows, top_k), torch.float32, dev, stream)
    _need(cand_ids, "cand_ids", torch.int64)
    _need(cand_u, "cand_u", torch.float32)
    if workspace is None:
        workspace = _workspace(unary_topk_workspace_size(rows, draft_vocab, top_k,
                                                         code), dev, stream)
    if err is None:
        err = _error_word(dev, stream)
    _check("dflash2_unary_topk", library().dflash2_unary_topk(
        _ptr(h), _ptr(lm_head), rows, hidden, draft_vocab, target_vocab, float(mult),
        float(cap), top_k, code, _ptr(cand_ids), _ptr(cand_u), _ptr(workspace),
        workspace.numel(), _ptr(err), _stream(stream)))
    return cand_ids, cand_u, err


def quantize_rows_e4m3(x, q=None, scale=None, stream=None):
    """dflash2_quantize_rows_e4m3: per-row E4M3 codes (uint8) and scales of x."""
    rows, cols = x.shape
    _need(x, "x")
    if q is None:
        q = _empty((rows, cols), torch.uint8, x.device, stream)
    if scale is None:
        scale = _empty(rows, torch.float32, x.device, stream)
    _check("dflash2_quantize_rows_e4m3", library().dflash2_quantize_rows_e4m3(
        _ptr(x), rows, cols, _dtype_code(x), _ptr(q), _ptr(scale), _stream(stream)))
    return q, scale


def unary_topk_fp8_workspace_size(rows: int, hidden: int, draft_vocab: int, top_k: int) -> int:
    return int(library().dflash2_unary_topk_fp8_workspace_size(rows, hidden, draft_vocab, top_k))


def unary_topk_fp8(h, lm_head_q, w_scale, target_vocab: int, mult: float, cap: float, top_k: int,
                   cand_ids=None, cand_u=None, workspace=None, err=None, stream=None):
    """dflash2_unary_topk_fp8: top_k (ids, u) per row of h against an E4M3 head
    (lm_head_q uint8 codes [draft_vocab, hidden], w_scale float [draft_vocab])."""
    rows, hidden = h.shape
    draft_vocab = lm_head_q.shape[0]
    _need(h, "h")
    _need(lm_head_q, "lm_head_q", torch.uint8, (draft_vocab, hidden))
    _need(w_scale, "w_scale", torch.float32, (draft_vocab,))
    dev = h.device
    if cand_ids is None:
        cand_ids = _empty((rows, top_k), torch.int64, dev, stream)
    if cand_u is None:
        cand_u = _empty((rows, top_k), torch.float32, dev, stream)
    if workspace is None:
        workspace = _workspace(unary_topk_fp8_workspace_size(rows, hidden, draft_vocab,
                                                             top_k), dev, stream)
    if err is None:
        err = _error_word(dev, stream)
    _check("dflash2_unary_topk_fp8", library().dflash2_unary_topk_fp8(
        _ptr(h), _dtype_code(h), _ptr(lm_head_q), _ptr(w_scale), rows, hidden, draft_vocab,
        target_vocab, float(mult), float(cap), top_k, _ptr(cand_ids), _ptr(cand_u),
        _ptr(workspace), workspace.numel(), _ptr(err), _stream(stream)))
    return cand_ids, cand_u, err


def quantize_rows_nvfp4(x, codes=None, scales=None, g=None, stream=None):
    """dflash2_quantize_rows_nvfp4: per-row NVFP4 codes (uint8, two per byte),
    E4M3 block scales (uint8, one per 16 elements) and fp32 second-level
    scales of x."""
    rows, cols = x.shape
    _need(x, "x")
    dev = x.device
    if codes is None:
        codes = _empty((rows, cols // 2), torch.uint8, dev, stream)
    if scales is None:
        scales = _empty((rows, cols // 16), torch.uint8, dev, stream)
    if g is None:
        g = _empty(rows, torch.float32, dev, stream)
    _check("dflash2_quantize_rows_nvfp4", library().dflash2_quantize_rows_nvfp4(
        _ptr(x), rows, cols, _dtype_code(x), _ptr(codes), _ptr(scales), _ptr(g),
        _stream(stream)))
    return codes, scales, g


def nvfp4_tile_scales(scales, hidden: int, tiles=None, stream=None):
    """dflash2_nvfp4_tile_scales: the scale tiles of row-major E4M3 block
    scales [rows, hidden / 16] (uint8), as the NVFP4 GEMM reads them."""
    rows = scales.shape[0]
    _need(scales, "scales", torch.uint8, (rows, hidden // 16))
    if tiles is None:
        tiles = _workspace(int(library().dflash2_nvfp4_scale_tiles_size(rows, hidden)),
                           scales.device, stream)
    _check("dflash2_nvfp4_tile_scales", library().dflash2_nvfp4_tile_scales(
        _ptr(scales), rows, hidden, _ptr(tiles), _stream(stream)))
    return tiles


def unary_topk_nvfp4_workspace_size(rows: int, hidden: int, draft_vocab: int, top_k: int) -> int:
    return int(library().dflash2_unary_topk_nvfp4_workspace_size(rows, hidden, draft_vocab,
                                                                 top_k))


def unary_topk_nvfp4(h, lm_head_q, w_scale_tiles, w_global: float, target_vocab: int, mult: float,
                     cap: float, top_k: int, cand_ids=None, cand_u=None, workspace=None, err=None,
                     stream=None):
    """dflash2_unary_topk_nvfp4: top_k (ids, u) per row of h against an NVFP4
    head (lm_head_q uint8 [draft_vocab, hidden / 2] codes, w_scale_tiles its
    E4M3 block scales as nvfp4_tile_scales returns them, w_global its fp32
    scale)."""
    rows, hidden = h.shape
    draft_vocab = lm_head_q.shape[0]
    _need(h, "h")
    _need(lm_head_q, "lm_head_q", torch.uint8, (draft_vocab, hidden // 2))
    _need(w_scale_tiles, "w_scale_tiles", torch.uint8)
    need = int(library().dflash2_nvfp4_scale_tiles_size(draft_vocab, hidden))
    if w_scale_tiles.numel() < need:
        raise ValueError(f"w_scale_tiles: uint8 scale tiles of {need} bytes expected")
    dev = h.device
    if cand_ids is None:
        cand_ids = _empty((rows, top_k), torch.int64, dev, stream)
    if cand_u is None:
        cand_u = _empty((rows, top_k), torch.float32, dev, stream)
    if workspace is None:
        workspace = _workspace(unary_topk_nvfp4_workspace_size(rows, hidden, draft_vocab,
                                                               top_k), dev, stream)
    if err is None:
        err = _error_word(dev, stream)
    _check("dflash2_unary_topk_nvfp4", library().dflash2_unary_topk_nvfp4(
        _ptr(h), _dtype_code(h), _ptr(lm_head_q), _ptr(w_scale_tiles), float(w_global), rows, hidden,
        draft_vocab, target_vocab, float(mult), float(cap), top_k, _ptr(cand_ids), _ptr(cand_u),
        _ptr(workspace), workspace.numel(), _ptr(err), _stream(stream)))
    return cand_ids, cand_u, err


def topk_merge(ids, u, id_offsets, k_out: int, out_ids=None, out_u=None, err=None, stream=None):
    """dflash2_topk_merge: the k_out best (u, global id) per row over shard
    lists ids / u [shards, rows, k_in] (shard-local ids; u = -inf absent)."""
    shards, rows, k_in = ids.shape
    _need(ids, "ids", torch.int64)
    _need(u, "u", torch.float32, tuple(ids.shape))
    offs = [int(o) for o in id_offsets]
    if len(offs) != shards:
        raise ValueError("one id offset per shard")
    dev = ids.device
    if out_ids is None:
        out_ids = _empty((rows, k_out), torch.int64, dev, stream)
    if out_u is None:
        out_u = _empty((rows, k_out), torch.float32, dev, stream)
    _need(out_ids, "out_ids", torch.int64, (rows, k_out))
    _need(out_u, "out_u", torch.float32, (rows, k_out))
    if err is None:
        err = _error_word(dev, stream)
    host_offs = (ctypes.c_int64 * shards)(*offs)
    _check("dflash2_topk_merge", library().dflash2_topk_merge(
        _ptr(ids), _ptr(u), ctypes.cast(host_offs, ctypes.c_void_p), shards, rows, k_in, k_out,
        _ptr(out_ids), _ptr(out_u), _ptr(err), _stream(stream)))
    return out_ids, out_u, err


def vocab_shard(draft_vocab: int, target_vocab: int, shards: int, s: int):
    """Shard s of `shards` near-equal slices of the lm_head rows: (first id,
    rows in the slice, ids of the slice below target_vocab)."""
    if not 0 <= s < shards:
        raise ValueError("shard index out of range")
    per = -(-draft_vocab // shards)
    first = min(s * per, draft_vocab)
    n = min(per, draft_vocab - first)
    return first, n, max(0, min(n, target_vocab - first))


def shard_topk(h, lm_head_slice, first: int, target_vocab: int, mult: float, cap: float,
               top_k: int, workspace=None, err=None, stream=None):
    """This shard's part of a vocab-sharded unary top-K: dflash2_unary_topk over
    its lm_head rows, as a [rows, top_k] list with shard-local ids.  A slice
    with fewer than top_k ids below target_vocab pads its list with u = -inf
    (absent for the merge)."""
    rows = h.shape[0]
    n = lm_head_slice.shape[0]
    local_target = max(0, min(n, target_vocab - first))
    k_here = min(top_k, local_target)
    if k_here == top_k:
        ids, u, _ = unary_topk(h, lm_head_slice, local_target, mult, cap, top_k,
                               workspace=workspace, err=err, stream=stream)
        return ids, u
    s = torch.cuda.current_stream(h.device) if stream is None else stream
    with torch.cuda.stream(s):
        ids = torch.zeros((rows, top_k), dtype=torch.int64, device=h.device)
        u = torch.full((rows, top_k), float("-inf"), dtype=torch.float32, device=h.device)
        if k_here > 0 and rows > 0:
            i2, u2, _ = unary_topk(h, lm_head_slice, local_target, mult, cap, k_here,
                                   workspace=workspace, err=err, stream=s)
            ids[:, :k_here] = i2
            u[:, :k_here] = u2
    return ids, u


def gather_shard_lists(ids, u, group=None):
    """The exchange of a vocab-sharded top-K: every rank's [rows, K] list,
    all-gathered into [world, rows, K] (rank order = shard order)."""
    import torch.distributed as dist
    world = dist.get_world_size(group)
    all_ids = [torch.empty_like(ids) for _ in range(world)]
    all_u = [torch.empty_like(u) for _ in range(world)]
    dist.all_gather(all_ids, ids.contiguous(), group=group)
    dist.all_gather(all_u, u.contiguous(), group=group)
    return torch.stack(all_ids), torch.stack(all_u)


def unary_topk_vocab_sharded(h, lm_head_slice, draft_vocab: int, target_vocab: int, mult: float,
                             cap: float, top_k: int, group=None, err=None, stream=None):
    """Vocab-sharded unary top-K over a process group: this rank holds lm_head
    rows vocab_shard(draft_vocab, target_vocab, world, rank); the shard's
    list, one all-gather and dflash2_topk_merge give every rank the unsharded
    result (the same ids and u as dflash2_unary_topk over the whole lm_head)."""
    import torch.distributed as dist
    world, rank = dist.get_world_size(group), dist.get_rank(group)
    first, n, _ = vocab_shard(draft_vocab, target_vocab, world, rank)
    if lm_head_slice.shape[0] != n:
        raise ValueError(f"rank {rank} holds {lm_head_slice.shape[0]} lm_head rows, expected {n}")
    ids, u = shard_topk(h, lm_head_slice, first, target_vocab, mult, cap, top_k, err=err,
                        stream=stream)
    all_ids, all_u = gather_shard_lists(ids, u, group)
    offsets = [vocab_shard(draft_vocab, target_vocab, world, s)[0] for s in range(world)]
    return topk_merge(all_ids, all_u, offsets, top_k, err=err, stream=stream)


def selector_walk_workspace_size(batch: int, slots: int, hidden: int, rank: int, top_k: int,
                                 dtype_code: int) -> int:
    return int(library().dflash2_selector_walk_workspace_size(batch, slots, hidden, rank, top_k,
                                                              dtype_code))


def selector_walk(h, proj, A, B, anchor_ids, cand_ids, cand_u, temperatures, greedy, uniforms,
                  tokens=None, q=None, path_scores=None, workspace=None, err=None,
                  with_path_scores: bool = False, stream=None):
    """dflash2_selector_walk over [batch, slots, top_k] candidates."""
    batch, slots, top_k = cand_ids.shape
    hidden = h.shape[-1]
    rank = proj.shape[0]
    code = _dtype_code(h)
    dev = h.device
    for t, nm in ((h, "h"), (proj, "proj"), (A, "A"), (B, "B")):
        _need(t, nm, h.dtype)
    _need(anchor_ids, "anchor_ids", torch.int64, (batch,))
    _need(cand_ids, "cand_ids", torch.int64)
    _need(cand_u, "cand_u", torch.float32, (batch, slots, top_k))
    _need(temperatures, "temperatures", torch.float32, (batch,))
    _need(greedy, "greedy", torch.uint8, (batch,))
    _need(uniforms, "uniforms", torch.float32, (batch, slots))
    if A.shape != B.shape or A.shape[1] != rank:
        raise ValueError("A and B must both be [table_rows, rank]")
    if tokens is None:
        tokens = _empty((batch, slots), torch.int64, dev, stream)
    if q is None:
        q = _empty((batch, slots, top_k), torch.float32, dev, stream)
    if path_scores is None and with_path_scores:
        path_scores = _empty((batch, slots, top_k), torch.float32, dev, stream)
    if workspace is None:
        workspace = _workspace(selector_walk_workspace_size(batch, slots, hidden, rank, top_k,
                                                            code), dev, stream)
    if err is None:
        err = _error_word(dev, stream)
    _check("dflash2_selector_walk", library().dflash2_selector_walk(
        _ptr(h), _ptr(proj), _ptr(A), _ptr(B), A.shape[0], _ptr(anchor_ids), _ptr(cand_ids),
        _ptr(cand_u), _ptr(temperatures), _ptr(greedy), _ptr(uniforms), batch, slots, hidden,
        rank, top_k, code, _ptr(tokens), _ptr(q), _ptr(path_scores), _ptr(workspace),
        workspace.numel(), _ptr(err), _stream(stream)))
    return tokens, q, path_scores, err


def selector_project(h, proj, batch: int, slots: int, top_k: int, workspace, err=None,
                     stream=None):
    """dflash2_selector_project: the projection partials of g = h . proj^T into
    `workspace` (a selector_walk workspace for the same shapes), for a later
    selector_walk_projected call ordered after it."""
    hidden = h.shape[-1]
    rank = proj.shape[0]
    code = _dtype_code(h)
    for t, nm in ((h, "h"), (proj, "proj")):
        _need(t, nm, h.dtype)
    if h.numel() != batch * slots * hidden:
        raise ValueError("h must hold batch * slots rows of hidden")
    _need(workspace, "workspace", torch.uint8)
    _check("dflash2_selector_project", library().dflash2_selector_project(
        _ptr(h), _ptr(proj), batch, slots, hidden, rank, top_k, code, _ptr(workspace),
        workspace.numel(), _ptr(err), _stream(stream)))
    return workspace


def selector_walk_projected(A, B, anchor_ids, cand_ids, cand_u, temperatures, greedy, uniforms,
                            hidden: int, workspace, tokens=None, q=None, path_scores=None,
                            err=None, with_path_scores: bool = False, stream=None):
    """dflash2_selector_walk_projected: the edges and the walk from the
    projection a selector_project call left in `workspace`."""
    batch, slots, top_k = cand_ids.shape
    rank = A.shape[1]
    code = _dtype_code(A)
    dev = A.device
    _need(A, "A")
    _need(B, "B", A.dtype)
    _need(anchor_ids, "anchor_ids", torch.int64, (batch,))
    _need(cand_ids, "cand_ids", torch.int64)
    _need(cand_u, "cand_u", torch.float32, (batch, slots, top_k))
    _need(temperatures, "temperatures", torch.float32, (batch,))
    _need(greedy, "greedy", torch.uint8, (batch,))
    _need(uniforms, "uniforms", torch.float32, (batch, slots))
    _need(workspace, "workspace", torch.uint8)
    if A.shape != B.shape:
        raise ValueError("A and B must both be [table_rows, rank]")
    if tokens is None:
        tokens = _empty((batch, slots), torch.int64, dev, stream)
    if q is None:
        q = _empty((batch, slots, top_k), torch.float32, dev, stream)
    if path_scores is None and with_path_scores:
        path_scores = _empty((batch, slots, top_k), torch.float32, dev, stream)
    if err is None:
        err = _error_word(dev, stream)
    _check("dflash2_selector_walk_projected", library().dflash2_selector_walk_projected(
        _ptr(A), _ptr(B), A.shape[0], _ptr(anchor_ids), _ptr(cand_ids), _ptr(cand_u),
        _ptr(temperatures), _ptr(greedy), _ptr(uniforms), batch, slots, hidden, rank, top_k, code,
        _ptr(tokens), _ptr(q), _ptr(path_scores), _ptr(workspace), workspace.numel(), _ptr(err),
        _stream(stream)))
    return tokens, q, path_scores, err


def selector_walk_noalloc(h, proj, A, B, anchor_ids, cand_ids, cand_u, temperatures, greedy,
                          uniforms, tokens=None, q=None, path_scores=None, err=None,
                          with_path_scores: bool = False, stream=None):
    """dflash2_selector_walk_noalloc: the selector walk with the library's own
    fixed 4 MiB scratch instead of a workspace, for callers that cannot hand
    over device memory at call time.  Calls that overlap on the GPU share that
    scratch and race; shapes needing more scratch raise Dflash2Error."""
    batch, slots, top_k = cand_ids.shape
    for t, nm in ((h, "h"), (proj, "proj"), (A, "A"), (B, "B")):
        _need(t, nm, h.dtype)
    _need(anchor_ids, "anchor_ids", torch.int64, (batch,))
    _need(cand_ids, "cand_ids", torch.int64)
    _need(cand_u, "cand_u", torch.float32, (batch, slots, top_k))
    _need(temperatures, "temperatures", torch.float32, (batch,))
    _need(greedy, "greedy", torch.uint8, (batch,))
    _need(uniforms, "uniforms", torch.float32, (batch, slots))
    dev = h.device
    if tokens is None:
        tokens = _empty((batch, slots), torch.int64, dev, stream)
    if q is None:
        q = _empty((batch, slots, top_k), torch.float32, dev, stream)
    if path_scores is None and with_path_scores:
        path_scores = _empty((batch, slots, top_k), torch.float32, dev, stream)
    if err is None:
        err = _error_word(dev, stream)
    _check("dflash2_selector_walk_noalloc", library().dflash2_selector_walk_noalloc(
        _ptr(h), _ptr(proj), _ptr(A), _ptr(B), A.shape[0], _ptr(anchor_ids), _ptr(cand_ids),
        _ptr(cand_u), _ptr(temperatures), _ptr(greedy), _ptr(uniforms), batch, slots,
        h.shape[-1], proj.shape[0], top_k, _dtype_code(h), _ptr(tokens), _ptr(q),
        _ptr(path_scores), _ptr(err), _stream(stream)))
    return tokens, q, path_scores, err


def d2t_remap(draft_ids, d2t, draft_vocab: int, target_vocab: int, out=None, err=None,
              stream=None):
    """dflash2_d2t_remap: target = draft + d2t[draft] (identity when d2t is None)."""
    _need(draft_ids, "draft_ids", torch.int64)
    if d2t is not None:
        _need(d2t, "d2t", torch.int64, (draft_vocab,))
    if out is None:
        out = _empty(draft_ids.shape, draft_ids.dtype, draft_ids.device, stream)
    if err is None:
        err = _error_word(draft_ids.device, stream)
    _check("dflash2_d2t_remap", library().dflash2_d2t_remap(
        _ptr(draft_ids), _ptr(d2t), draft_ids.numel(), draft_vocab, target_vocab, _ptr(out),
        _ptr(err), _stream(stream)))
    return out, err


def conv_prepare(x, w_kp, base2, block_size: int, group_size: int, taps: int, out=None,
                 coef=None, err=None, stream=None):
    """dflash2_conv_prepare: (conv of x with coefficient side 0, coef [n, 2, taps, groups])."""
    n, hidden = x.shape
    groups = hidden // group_size
    code = _dtype_code(x)
    _need(x, "x", x.dtype)
    _need(w_kp, "w_kp", x.dtype, (2 * taps * groups, hidden))
    _need(base2, "base2", x.dtype, (2, taps, hidden))
    if out is None:
        out = _empty(x.shape, x.dtype, x.device, stream)
    if coef is None:
        coef = _empty((n, 2, taps, groups), x.dtype, x.device, stream)
    _need(coef, "coef", x.dtype, (n, 2, taps, groups))
    if err is None:
        err = _error_word(x.device, stream)
    _check("dflash2_conv_prepare", library().dflash2_conv_prepare(
        _ptr(x), _ptr(w_kp), _ptr(base2), n, hidden, group_size, taps, block_size, code,
        _ptr(out), _ptr(coef), _ptr(err), _stream(stream)))
    return out, coef, err


def conv_finish(y, coef, base2, block_size: int, group_size: int, taps: int, out=None,
                stream=None):
    """dflash2_conv_finish: conv of y with coefficient side 1 and base side 1."""
    n, hidden = y.shape
    groups = hidden // group_size
    code = _dtype_code(y)
    _need(y, "y", y.dtype)
    _need(coef, "coef", y.dtype, (n, 2, taps, groups))
    _need(base2, "base2", y.dtype, (2, taps, hidden))
    if out is None:
        out = _empty(y.shape, y.dtype, y.device, stream)
    _check("dflash2_conv_finish", library().dflash2_conv_finish(
        _ptr(y), _ptr(base2), _ptr(coef), n, hidden, group_size, taps, block_size, code,
        _ptr(out), _stream(stream)))
    return out


def verify(target_logits, temperatures, greedy, draft, cand, q, uniforms, accept_len=None,
           out_tokens=None, workspace=None, err=None, stream=None):
    """dflash2_verify: speculative-sampling verification of a proposed block.

    target_logits [B, S+1, V]; draft [B, S] and cand [B, S, K] are target ids."""
    b, s1, vocab = target_logits.shape
    slots = s1 - 1
    k = cand.shape[-1]
    code = _dtype_code(target_logits)
    _need(target_logits, "target_logits", target_logits.dtype)
    _need(temperatures, "temperatures", torch.float32, (b,))
    _need(greedy, "greedy", torch.uint8, (b,))
    _need(draft, "draft", torch.int64, (b, slots))
    _need(cand, "cand", torch.int64, (b, slots, k))
    _need(q, "q", torch.float32, (b, slots, k))
    _need(uniforms, "uniforms", torch.float32, (b, s1))
    dev = target_logits.device
    if accept_len is None:
        accept_len = _empty(b, torch.int64, dev, stream)
    if out_tokens is None:
        out_tokens = _empty((b, s1), torch.int64, dev, stream)
    if workspace is None:
        workspace = _workspace(verify_workspace_size(b, slots, vocab), dev, stream)
    if err is None:
        err = _error_word(dev, stream)
    _check("dflash2_verify", library().dflash2_verify(
        _ptr(target_logits), vocab, _ptr(temperatures), _ptr(greedy), _ptr(draft), _ptr(cand),
        _ptr(q), _ptr(uniforms), b, slots, k, code, _ptr(accept_len), _ptr(out_tokens),
        _ptr(workspace), workspace.numel(), _ptr(err), _stream(stream)))
    return accept_len, out_tokens, err


def verify_workspace_size(batch: int, slots: int, vocab: int) -> int:
    return int(library().dflash2_verify_workspace_size(batch, slots, vocab))


def philox_uniforms(seed: int, n: int, out=None, offset: int = 0, counter=None, device=None,
                    stream=None):
    """dflash2_philox_uniforms: n float32 uniforms in [0, 1) from Philox4x64-10.

    With ``counter`` (a 1-element int64 device tensor holding the uint64 bits),
    the base is read and advanced on the device, so a captured graph draws a
    fresh sequence at every replay."""
    if counter is not None:
        _need(counter, "counter", torch.int64, (1,))
        device = counter.device
    if out is None:
        if device is None:
            raise ValueError("philox_uniforms needs `out`, `counter` or `device`")
        out = _empty(int(n), torch.float32, device, stream)
    else:
        _need(out, "out", torch.float32)
        if out.numel() < n:
            raise ValueError("out holds fewer than n elements")
    _check("dflash2_philox_uniforms", library().dflash2_philox_uniforms(
        int(seed) & (2**64 - 1), int(offset) & (2**64 - 1), _ptr(counter), int(n), _ptr(out),
        _stream(stream)))
    return out


# ---- paged key/value cache and attention ----------------------------------------------

class KVCache(NamedTuple):
    """One layer's paged cache: keys and values [pages, kv_heads, page_size,
    head_dim], in float32 or bfloat16, or as uint8 E4M3 codes with one exponent
    byte per row in k_exp and v_exp [pages, kv_heads, page_size], 79 to 175 (the
    nearest of these is taken for others).  A slot is page * page_size + offset.
    The tensors are the caller's."""
    k: torch.Tensor
    v: torch.Tensor
    k_exp: torch.Tensor | None = None
    v_exp: torch.Tensor | None = None

    @property
    def e4m3(self) -> bool:
        return self.k.dtype == torch.uint8


def new_kv_cache(pages: int, page_size: int, kv_heads: int, head_dim: int,
                 dtype=torch.bfloat16, e4m3: bool = False, device="cuda") -> KVCache:
    """An empty cache: rows in `dtype`, or E4M3 codes and exponents.  What is
    not written yet holds zeros."""
    shape = (pages, kv_heads, page_size, head_dim)
    held = torch.uint8 if e4m3 else dtype
    k, v = (torch.zeros(shape, dtype=held, device=device) for _ in range(2))
    if not e4m3:
        return KVCache(k, v)
    return KVCache(k, v, *(torch.full(shape[:3], 127, dtype=torch.uint8, device=device)
                           for _ in range(2)))


def _need_rows(t: torch.Tensor, name: str, dtype, shape) -> int:
    """A [tokens, heads, head_dim] tensor whose tokens may be strided (a slice
    of a packed projection) with contiguous heads; returns the token stride."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    n, heads, d = shape
    st = t.stride()
    if st[2] == 1 and st[1] == d and n > 1 and st[0] >= heads * d:
        return st[0]
    if (st[2] != 1 and d > 1) or (st[1] != d and heads > 1):
        raise ValueError(f"{name} must have contiguous heads")
    if n > 1 and st[0] < heads * d:
        raise ValueError(f"{name} must not repeat tokens")
    return st[0] if n > 1 else heads * d


def _need_error_word(err, device, stream):
    if err is None:
        return _error_word(device, stream)
    if not (err.is_cuda and err.dtype == torch.int32 and err.numel()):
        _need(err, "err", torch.int32)
        raise ValueError("err must hold a word")
    return err


def _need_cache(c: KVCache, dtype):
    k, v, k_exp, v_exp = c
    shape = k.shape
    pages, heads, ps, d = shape
    if k.dtype == torch.uint8:
        if k_exp is None or v_exp is None:
            raise ValueError("an E4M3 cache needs k_exp and v_exp")
        _need(k, "cache.k", torch.uint8)
        _need(v, "cache.v", torch.uint8, shape)
        exps = (pages, heads, ps)
        _need(k_exp, "cache.k_exp", torch.uint8, exps)
        _need(v_exp, "cache.v_exp", torch.uint8, exps)
        return pages, heads, ps, d, KV_E4M3
    _need(k, "cache.k", dtype)
    _need(v, "cache.v", dtype, shape)
    return pages, heads, ps, d, KV_NATIVE


def kv_cache_write(cache: KVCache, k, v, slots, err=None, stream=None):
    """dflash2_kv_cache_write: keys and values [n, kv_heads, head_dim] into
    their slots (int64 [n], negative skips); an E4M3 cache is quantised on the
    way.  k and v may be slices of a packed projection."""
    pages, heads, ps, d, fmt = _need_cache(cache, k.dtype)
    n = k.shape[0]
    ks = _need_rows(k, "k", k.dtype, (n, heads, d))
    vs = _need_rows(v, "v", k.dtype, (n, heads, d))
    _need(slots, "slots", torch.int64, (n,))
    err = _need_error_word(err, k.device, stream)
    _check("dflash2_kv_cache_write", library().dflash2_kv_cache_write(
        _ptr(k), _ptr(v), ks, vs, _ptr(slots), n, heads, d, ps, pages, _dtype_code(k), fmt,
        _ptr(cache.k), _ptr(cache.v), _ptr(cache.k_exp), _ptr(cache.v_exp), _ptr(err),
        _stream(stream)))
    return err


def kv_cache_read(cache: KVCache, slots, dtype=torch.bfloat16, k_out=None, v_out=None, err=None,
                  stream=None):
    """dflash2_kv_cache_read: the rows at `slots` (int64 [n], negative gives
    zeros) as keys and values [n, kv_heads, head_dim] in `dtype`."""
    pages, heads, ps, d, fmt = _need_cache(cache, dtype)
    _need(slots, "slots", torch.int64)
    n = slots.numel()
    if k_out is None:
        k_out = _empty((n, heads, d), dtype, slots.device, stream)
    else:
        _need(k_out, "k_out", dtype, (n, heads, d))
    if v_out is None:
        v_out = _empty(k_out.shape, k_out.dtype, k_out.device, stream)
    else:
        _need(v_out, "v_out", dtype, (n, heads, d))
    err = _need_error_word(err, slots.device, stream)
    _check("dflash2_kv_cache_read", library().dflash2_kv_cache_read(
        _ptr(cache.k), _ptr(cache.v), _ptr(cache.k_exp), _ptr(cache.v_exp), _ptr(slots), n, heads,
        d, ps, pages, _dtype_code(k_out), fmt, _ptr(k_out), _ptr(v_out), _ptr(err),
        _stream(stream)))
    return k_out, v_out, err


def tree_attention_workspace_size(total_q: int, batch: int, q_heads: int, kv_heads: int,
                                  head_dim: int) -> int:
    return int(library().dflash2_tree_attention_workspace_size(total_q, batch, q_heads, kv_heads,
                                                               head_dim))


def tree_attention(q, cache: KVCache, page_table, cu_q, kv_lens, scale: float, tree_mask=None,
                   out=None, lse=None, with_lse: bool = False, workspace=None, err=None,
                   stream=None):
    """dflash2_tree_attention: drafted tokens' queries q [total_q, q_heads,
    head_dim] (tokens may be strided) over the paged cache, which already
    holds their keys and values as each request's last cu_q[b + 1] - cu_q[b]
    of kv_lens[b] positions (page_table int32 [batch, max_pages]).  tree_mask
    int64 [total_q, words]: bit j of a row, it sees node j; None, a chain.
    Returns (out, lse or None, err)."""
    total, heads, d = q.shape
    pages, kv_heads, ps, kd, fmt = _need_cache(cache, q.dtype)
    if kd != d:
        raise ValueError(f"q has head_dim {d}, the cache {kd}")
    batch, max_pages = page_table.shape
    qs = _need_rows(q, "q", q.dtype, (total, heads, d))
    _need(page_table, "page_table", torch.int32)
    _need(cu_q, "cu_q", torch.int32, (batch + 1,))
    _need(kv_lens, "kv_lens", torch.int32, (batch,))
    words = 0
    if tree_mask is not None:
        words = tree_mask.shape[-1]
        _need(tree_mask, "tree_mask", torch.int64, (total, words))
        if words < 1:  # an empty tensor's pointer is NULL: no mask
            raise ValueError("tree_mask must have a word per token at least")
    dev = q.device
    if out is None:
        out = _empty((total, heads, d), q.dtype, dev, stream)
    else:
        _need(out, "out", q.dtype, (total, heads, d))
    if lse is not None:
        _need(lse, "lse", torch.float32, (total, heads))
    elif with_lse:
        lse = _empty((total, heads), torch.float32, dev, stream)
    if workspace is None:
        workspace = _workspace(tree_attention_workspace_size(total, batch, heads, kv_heads,
                                                             d), dev, stream)
    else:
        _need(workspace, "workspace")
    err = _need_error_word(err, dev, stream)
    _check("dflash2_tree_attention", library().dflash2_tree_attention(
        _ptr(q), qs, _ptr(cache.k), _ptr(cache.v), _ptr(cache.k_exp), _ptr(cache.v_exp),
        _ptr(page_table), max_pages, pages, ps, _ptr(cu_q), _ptr(kv_lens), _ptr(tree_mask), words,
        batch, total, heads, kv_heads, d, float(scale), _dtype_code(q), fmt, _ptr(out), _ptr(lse),
        _ptr(workspace), workspace.nbytes, _ptr(err), _stream(stream)))
    return out, lse, err


def prompt_attention_workspace_size(total_q: int, batch: int, q_heads: int, kv_heads: int,
                                    head_dim: int) -> int:
    return int(library().dflash2_prompt_attention_workspace_size(total_q, batch, q_heads, kv_heads,
                                                                 head_dim))


def prompt_attention(q, k, v, cu_q, scale: float, out=None, lse=None, with_lse: bool = False,
                     workspace=None, err=None, stream=None):
    """dflash2_prompt_attention: causal attention of packed prompts, q
    [total_q, q_heads, head_dim], k and v [total_q, kv_heads, head_dim] (slices
    of one packed projection are read in place), request b the tokens cu_q[b]
    .. cu_q[b + 1] - 1.  Returns (out, lse or None, err)."""
    total, heads, d = q.shape
    kv_heads = k.shape[1]
    qs = _need_rows(q, "q", q.dtype, (total, heads, d))
    ks = _need_rows(k, "k", q.dtype, (total, kv_heads, d))
    vs = _need_rows(v, "v", q.dtype, (total, kv_heads, d))
    _need(cu_q, "cu_q", torch.int32)
    batch = cu_q.numel() - 1
    if batch < 0:
        raise ValueError("cu_q must have batch + 1 entries")
    dev = q.device
    if out is None:
        out = _empty((total, heads, d), q.dtype, dev, stream)
    else:
        _need(out, "out", q.dtype, (total, heads, d))
    if lse is not None:
        _need(lse, "lse", torch.float32, (total, heads))
    elif with_lse:
        lse = _empty((total, heads), torch.float32, dev, stream)
    if workspace is None:
        workspace = _workspace(prompt_attention_workspace_size(total, batch, heads, kv_heads,
                                                               d), dev, stream)
    else:
        _need(workspace, "workspace")
    err = _need_error_word(err, dev, stream)
    _check("dflash2_prompt_attention", library().dflash2_prompt_attention(
        _ptr(q), _ptr(k), _ptr(v), qs, ks, vs, _ptr(cu_q), batch, total, heads, kv_heads, d,
        float(scale), _dtype_code(q), _ptr(out), _ptr(lse), _ptr(workspace), workspace.nbytes,
        _ptr(err), _stream(stream)))
    return out, lse, err


# ---- norms, FP8 linear layers and rotary positions -----------------------------------

def _need_matrix(t: torch.Tensor, name: str, dtype=None, shape=None) -> int:
    """A [rows, cols] tensor whose rows may be strided (a slice of a wider one); returns
    the row stride."""
    if (t.is_cuda and (dtype is None or t.dtype == dtype) and t.dim() == 2
            and (shape is None or t.shape == shape)):
        rows, cols = t.shape
        s0, s1 = t.stride()
        if rows < 2 and (s1 == 1 or cols == 1):
            return cols
        if (s1 == 1 or cols == 1) and s0 >= cols:
            return s0
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or (shape is not None and t.shape != tuple(shape)):
        raise ValueError(f"{name} must have shape {'[rows, cols]' if shape is None else tuple(shape)}"
                         f", got {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    raise ValueError(f"{name} must not repeat rows")


_one_device = None  # whether there is but one: then every CUDA tensor lies on it


def _current_device() -> int:
    return torch._C._cuda_getDevice()


def _need_one_device(*tensors):
    """Everything a call is given lies on the current device, where it is launched."""
    global _one_device
    if _one_device:
        return
    if _one_device is None:
        _one_device = torch.cuda.device_count() == 1
    dev = _current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors must be on the current device cuda:{dev}, got {t.device}")


def _blocks_of(cols: int) -> int:
    return -(-cols // 128)


def quantize_blocks_e4m3(x, q=None, scale=None, stream=None):
    """dflash2_quantize_blocks_e4m3: E4M3 codes (uint8) of x [rows, cols] (rows may be
    strided) and one fp32 scale per 128 values of a row [rows, ceil(cols / 128)]."""
    xs = _need_matrix(x, "x")
    rows, cols = x.shape
    if q is None:
        q = _empty((rows, cols), torch.uint8, x.device, stream)
    else:
        _need(q, "q", torch.uint8, (rows, cols))
    if scale is None:
        scale = _empty((rows, _blocks_of(cols)), torch.float32, x.device, stream)
    else:
        _need(scale, "scale", torch.float32, (rows, _blocks_of(cols)))
    _need_one_device(x, q, scale)
    _check("dflash2_quantize_blocks_e4m3", library().dflash2_quantize_blocks_e4m3(
        _ptr(x), xs, rows, cols, _dtype_code(x), _ptr(q), _ptr(scale), _stream(stream)))
    return q, scale


def linear_fp8_blocks_workspace_size(rows: int, in_features: int, out_features: int) -> int:
    return int(library().dflash2_linear_fp8_blocks_workspace_size(rows, in_features, out_features))


def linear_fp8_blocks(x, w_q, w_scale, x_scale=None, out_dtype=None, out=None, workspace=None,
                      err=None, stream=None):
    """dflash2_linear_fp8_blocks: x [rows, in] times E4M3 weights w_q [out, in] (uint8)
    with a scale per 128 x 128 of them.  x is fp32 or bf16 (rows may be strided) and
    quantised on the way, or uint8 codes with their x_scale, as quantize_blocks_e4m3 or a
    norm here returns them.  out_dtype: x's, or bfloat16 for codes, unless given or `out`
    is.  Returns (out [rows, out], err)."""
    n_out, n_in = w_q.shape
    _need(w_q, "w_q", torch.uint8)
    _need(w_scale, "w_scale", torch.float32, (_blocks_of(n_out), _blocks_of(n_in)))
    rows = x.shape[0]
    dev = x.device
    codes = x.dtype == torch.uint8
    if codes:
        if x_scale is None:
            raise ValueError("codes need x_scale")
        _need(x, "x", torch.uint8, (rows, n_in))
        _need(x_scale, "x_scale", torch.float32, (rows, _blocks_of(n_in)))
    else:
        if x_scale is not None:
            raise ValueError("x_scale belongs to uint8 codes")
        xs = _need_matrix(x, "x", None, (rows, n_in))
        x_code = _dtype_code(x)
    if out is None:
        if out_dtype is None:
            out_dtype = torch.bfloat16 if codes else x.dtype
        out = _empty((rows, n_out), out_dtype, dev, stream)
    else:
        _need(out, "out", out_dtype, (rows, n_out))
    if workspace is not None:
        _need(workspace, "workspace")
    elif not codes:
        workspace = _workspace(linear_fp8_blocks_workspace_size(rows, n_in, n_out), dev, stream)
    err = _need_error_word(err, dev, stream)
    _need_one_device(x, w_q, w_scale, x_scale, out, workspace, err)
    _check("dflash2_linear_fp8_blocks", library().dflash2_linear_fp8_blocks(
        None if codes else _ptr(x), 0 if codes else xs, 0 if codes else x_code,
        _ptr(x) if codes else None, _ptr(x_scale), _ptr(w_q), _ptr(w_scale), rows, n_in, n_out,
        _dtype_code(out), _ptr(out), _ptr(workspace), 0 if workspace is None else workspace.nbytes,
        _ptr(err), _stream(stream)))
    return out, err


def _norm_out(rows, hidden, dtype, e4m3, out, scale, device, stream):
    if e4m3:
        if scale is None:
            scale = _empty((rows, _blocks_of(hidden)), torch.float32, device, stream)
        else:
            _need(scale, "scale", torch.float32, (rows, _blocks_of(hidden)))
    elif scale is not None:
        raise ValueError("scale belongs to e4m3=True")
    held = torch.uint8 if e4m3 else dtype
    if out is None:
        out = _empty((rows, hidden), held, device, stream)
    else:
        _need(out, "out", held, (rows, hidden))
    return out, scale


def sublayer_norm(x, weight, eps: float = 1e-6, weight_offset: float = 0.0, e4m3: bool = False,
                  out=None, scale=None, stream=None):
    """dflash2_sublayer_norm: rms(x) * (weight + weight_offset) of x [rows, hidden] (rows
    may be strided; fp32 or bf16, whatever weight is) in weight's dtype, or with e4m3 as
    codes and scales of E4M3 blocks.  Returns (out, scale or None)."""
    xs = _need_matrix(x, "x")
    rows, hidden = x.shape
    _need(weight, "weight", None, (hidden,))
    out, scale = _norm_out(rows, hidden, weight.dtype, e4m3, out, scale, x.device, stream)
    _need_one_device(x, weight, out, scale)
    _check("dflash2_sublayer_norm", library().dflash2_sublayer_norm(
        _ptr(x), xs, _dtype_code(x), _ptr(weight), float(weight_offset), float(eps), rows, hidden,
        _dtype_code(weight), _ptr(out), _ptr(scale), _stream(stream)))
    return out, scale


def sublayer_join(residual, y, post_weight=None, gate=None, gate_act: str = "none",
                  branch_scale: float = 1.0, next_weight=None, eps: float = 1e-6,
                  weight_offset: float = 0.0, e4m3: bool = False, residual_out=None, out=None,
                  scale=None, stream=None):
    """dflash2_sublayer_join: a sublayer's output y [rows, hidden] normed (post_weight),
    gated (gate [hidden], [rows, 1] or [rows, hidden]; gate_act none, sigmoid or tanh of
    it), scaled and added to residual, and the next sublayer's norm of that (next_weight),
    with e4m3 as E4M3 blocks.  The residual may have another dtype than y, the gate and
    the weights; residual_out may be residual.  Returns (residual_out, out or None, scale
    or None)."""
    rs = _need_matrix(residual, "residual")
    rows, hidden = residual.shape
    ys = _need_matrix(y, "y", None, (rows, hidden))
    dt, dev = y.dtype, y.device
    for w, name in ((post_weight, "post_weight"), (next_weight, "next_weight")):
        if w is not None:
            _need(w, name, dt, (hidden,))
    kind, gs = GATE_NONE, 0
    if gate_act not in GATE_ACTS:
        raise ValueError(f"gate_act must be one of {', '.join(GATE_ACTS)}, got {gate_act!r}")
    if gate is not None:
        if gate.dim() == 1:
            _need(gate, "gate", dt, (hidden,))
            kind = GATE_CHANNEL
        elif gate.dim() == 2 and gate.shape[1] == 1 and hidden > 1:
            gs = _need_matrix(gate, "gate", dt, (rows, 1))
            kind = GATE_TOKEN
        else:
            gs = _need_matrix(gate, "gate", dt, (rows, hidden))
            kind = GATE_FULL
    if residual_out is None:
        residual_out, ros = _empty((rows, hidden), residual.dtype, dev, stream), hidden
    else:
        ros = _need_matrix(residual_out, "residual_out", residual.dtype, (rows, hidden))
    if next_weight is not None:
        out, scale = _norm_out(rows, hidden, dt, e4m3, out, scale, dev, stream)
    elif out is not None or scale is not None or e4m3:
        raise ValueError("out, scale and e4m3 belong to next_weight")
    _need_one_device(residual, y, post_weight, gate, next_weight, residual_out, out, scale)
    _check("dflash2_sublayer_join", library().dflash2_sublayer_join(
        _ptr(residual), rs, _dtype_code(residual), _ptr(y), ys, _ptr(post_weight), _ptr(gate), kind,
        gs, GATE_ACTS[gate_act], float(branch_scale), _ptr(next_weight), float(weight_offset),
        float(eps), rows, hidden, _dtype_code(y), _ptr(residual_out), ros, _ptr(out), _ptr(scale),
        _stream(stream)))
    return residual_out, out, scale


class RotaryTable(NamedTuple):
    """Frequencies of rotary positions: freq int64 [rotary_dim / 2], the bits of a uint64
    fraction of a turn per position, in units of 2^-64; axis uint8 [rotary_dim / 2], the
    row of the positions that turns each pair; adjacent: pairs (2j, 2j + 1), not (j, j +
    rotary_dim / 2); magnitude: a factor of sines and cosines.  rotary_table makes one."""
    freq: torch.Tensor
    axis: torch.Tensor
    adjacent: bool = False
    magnitude: float = 1.0


def rotary_table(rotary_dim: int, base: float = 10000.0, sections=None, interleaved: bool = False,
                 inv_freq=None, adjacent: bool = False, magnitude: float = 1.0,
                 device="cuda") -> RotaryTable:
    """The table of frequencies base^(-2j / rotary_dim), or of inv_freq (radians per
    position, rotary_dim / 2 numbers).  sections: how many pairs each axis turns, adding
    up to rotary_dim / 2, one axis after the other; interleaved: the axes take turns from
    the first pair on, as far as each one's section goes, and the first axis takes the
    rest."""
    half = rotary_dim // 2
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and positive")
    if inv_freq is None:
        inv_freq = [float(base) ** (-j / half) for j in range(half)]
    inv_freq = [float(f) for f in inv_freq]
    sections = [half] if sections is None else [int(n) for n in sections]
    if len(inv_freq) != half or sum(sections) != half or min(sections) < 0 or len(sections) > 255:
        raise ValueError(f"inv_freq and sections must cover rotary_dim / 2 = {half} pairs")
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    if interleaved:
        axis = [0] * half
        for a, n in enumerate(sections[1:], 1):
            for i in range(n):
                if a + i * len(sections) >= half:
                    raise ValueError(f"section {a} does not fit between the others")
                axis[a + i * len(sections)] = a
    # the fraction of a turn, rounded to 2^-64; whole turns drop out
    turns = [round(math.fmod(f / math.tau, 1.0) * 2.0 ** 64) % 2 ** 64 for f in inv_freq]
    turns = [t - 2 ** 64 if t >= 2 ** 63 else t for t in turns]
    return RotaryTable(torch.tensor(turns, dtype=torch.int64, device=device),
                       torch.tensor(axis, dtype=torch.uint8, device=device), bool(adjacent),
                       float(magnitude))


def _need_rotary(positions, table: RotaryTable, n: int):
    freq, axis, adjacent, magnitude = table
    axes = 1 if positions.dim() == 1 else positions.shape[0]
    _need(positions, "positions", torch.int64, (n,) if positions.dim() == 1 else (axes, n))
    if not (freq.is_cuda and axis.is_cuda and freq.dtype == torch.int64 and axis.dtype == torch.uint8
            and freq.shape == axis.shape and freq.is_contiguous() and axis.is_contiguous()):
        _need(freq, "table.freq", torch.int64)
        _need(axis, "table.axis", torch.uint8, freq.shape)
    return (_ptr(positions), axes, _ptr(freq), _ptr(axis), 2 * freq.numel(),
            1 if adjacent else 0, magnitude)


def _rotated(x, name, out, stream):
    """The token strides of x and of where it goes, which is made unless given."""
    shape = x.shape
    xs = _need_rows(x, name, x.dtype, shape)
    if out is None:
        return xs, _empty(shape, x.dtype, x.device, stream), shape[1] * shape[2]
    return xs, out, _need_rows(out, name + "_out", x.dtype, shape)


def rotary(q, k, positions, table: RotaryTable, q_out=None, k_out=None, err=None, stream=None):
    """dflash2_rotary: queries q [n, q_heads, head_dim] and keys k [n, kv_heads, head_dim]
    (slices of a packed projection are read in place; k may be None) turned by positions
    int64 [n] or [axes, n].  q_out and k_out may be q and k.  Returns (q_out, k_out or
    None, err)."""
    n, heads, d = q.shape
    place = _need_rotary(positions, table, n)
    qs, q_out, qos = _rotated(q, "q", q_out, stream)
    ks = kos = kv_heads = 0
    if k is not None:
        kv_heads = k.shape[1]
        if k.shape != (n, kv_heads, d) or k.dtype != q.dtype:
            raise ValueError(f"k must be {q.dtype} [{n}, kv_heads, {d}]")
        ks, k_out, kos = _rotated(k, "k", k_out, stream)
    elif k_out is not None:
        raise ValueError("k_out without k")
    err = _need_error_word(err, q.device, stream)
    _need_one_device(q, k, positions, table.freq, table.axis, q_out, k_out, err)
    _check("dflash2_rotary", library().dflash2_rotary(
        _ptr(q), qs, _ptr(k), ks, *place, n, heads, kv_heads, d, _dtype_code(q), _ptr(q_out), qos,
        _ptr(k_out), kos, _ptr(err), _stream(stream)))
    return q_out, k_out, err


def rotary_kv_write(cache: KVCache, q, k, v, positions, table: RotaryTable, slots, q_out=None,
                    k_out=None, with_k: bool = False, err=None, stream=None):
    """dflash2_rotary_kv_write: rotary's turn of q (or None) and k, and the turned keys and
    the values v into the cache's slots (int64 [n], negative skips), an E4M3 cache's rows
    quantised on the way.  with_k: the turned keys are returned too (a prompt's own
    attention reads them).  Returns (q_out or None, k_out or None, err)."""
    pages, kv_heads, ps, d, fmt = _need_cache(cache, k.dtype)
    n = k.shape[0]
    if k.shape != (n, kv_heads, d):
        raise ValueError(f"k must have shape {(n, kv_heads, d)}, got {tuple(k.shape)}")
    place = _need_rotary(positions, table, n)
    ks = _need_rows(k, "k", k.dtype, (n, kv_heads, d))
    vs = _need_rows(v, "v", k.dtype, (n, kv_heads, d))
    _need(slots, "slots", torch.int64, (n,))
    qs = qos = kos = heads = 0
    if q is not None:
        heads = q.shape[1]
        if q.shape != (n, heads, d) or q.dtype != k.dtype:
            raise ValueError(f"q must be {k.dtype} [{n}, q_heads, {d}]")
        qs, q_out, qos = _rotated(q, "q", q_out, stream)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if with_k or k_out is not None:
        ks, k_out, kos = _rotated(k, "k", k_out, stream)
    err = _need_error_word(err, k.device, stream)
    _need_one_device(k, v, q, positions, table.freq, table.axis, slots, q_out, k_out, *cache, err)
    _check("dflash2_rotary_kv_write", library().dflash2_rotary_kv_write(
        _ptr(q), qs, _ptr(k), ks, _ptr(v), vs, *place, _ptr(slots), n, heads, kv_heads, d, ps,
        pages, _dtype_code(k), fmt, _ptr(q_out), qos, _ptr(k_out), kos, _ptr(cache.k),
        _ptr(cache.v), _ptr(cache.k_exp), _ptr(cache.v_exp), _ptr(err), _stream(stream)))
    return q_out, k_out, err


# ---- host <-> device helpers (plumbing) ----------------------------------------------

def to_device(a: np.ndarray, device) -> torch.Tensor:
    """numpy -> torch on `device`; uint16 arrays are bf16 bit patterns."""
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).to(device)
    return torch.from_numpy(np.ascontiguousarray(a)).to(device)


def to_host_bits(t: torch.Tensor) -> np.ndarray:
    """torch -> numpy; bf16 comes back as uint16 bit patterns."""
    t = t.detach().cpu().contiguous()
    if t.dtype == torch.bfloat16:
        return t.view(torch.int16).numpy().view(np.uint16)
    return t.numpy()


class ProposalBuffers:
    """Caller-owned outputs and workspaces of one proposal step (allocated once)."""

    def __init__(self, w, device):
        code = F32 if w.dtype == "f32" else BF16
        fdt = torch.float32 if w.dtype == "f32" else torch.bfloat16
        self.conv_out = torch.empty((w.n_tokens, w.hidden), dtype=fdt, device=device)
        self.cand_ids = torch.empty((w.rows, w.top_k), dtype=torch.int64, device=device)
        self.cand_u = torch.empty((w.rows, w.top_k), dtype=torch.float32, device=device)
        self.tokens = torch.empty((w.batch, w.slots), dtype=torch.int64, device=device)
        self.q = torch.empty((w.batch, w.slots, w.top_k), dtype=torch.float32, device=device)
        self.target_ids = torch.empty((w.batch, w.slots), dtype=torch.int64, device=device)
        self.uniforms = torch.empty((w.batch, w.slots), dtype=torch.float32, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.ws_topk = torch.empty(max(1, unary_topk_workspace_size(w.rows, w.draft_vocab, w.top_k, code)),
                                   dtype=torch.uint8, device=device)
        self.ws_walk = torch.empty(max(1, selector_walk_workspace_size(w.batch, w.slots, w.hidden,
                                                                       w.rank, w.top_k, code)),
                                   dtype=torch.uint8, device=device)
        # the second stream of an overlapped step and the events that fork it
        # from, and join it back into, the caller's stream
        self.side_stream = torch.cuda.Stream(device=device)
        self.fork = torch.cuda.Event()
        self.join = torch.cuda.Event()


def proposal_step(w, t: dict, bufs: ProposalBuffers | None = None, stream=None,
                  rng=None, overlap: bool = True) -> dict:
    """One pass of the hot path: conv, unary candidates, selector walk, d2t remap.

    `t` holds the device tensors of synth.make(w) (bf16 tensors as torch.bfloat16).
    With ``rng = (seed, counter)`` the walk's uniforms are drawn on the device
    (dflash2_philox_uniforms, counter advanced on the device) instead of taken
    from ``t["uniforms"]``.  Returns the output tensors (no synchronisation).

    With ``overlap`` the work that needs only the step's inputs (the uniforms,
    the grouped conv and the selector projection) runs on a second stream,
    forked from and joined back into `stream` by events, beside the unary
    top-K; the walk waits for both.  The results are the same either way; the
    fork and join are captured into a CUDA graph like the launches."""
    dev = t["h"].device
    if bufs is None:
        bufs = ProposalBuffers(w, dev)
    main = torch.cuda.current_stream(dev) if stream is None else stream
    side = main
    if overlap:
        side = bufs.side_stream
        bufs.fork.record(main)
        side.wait_event(bufs.fork)
    uniforms = t.get("uniforms")
    if rng is not None:
        seed, counter = rng
        philox_uniforms(seed, w.rows, out=bufs.uniforms.view(-1), counter=counter, stream=side)
        uniforms = bufs.uniforms
    grouped_conv(t["x"], t["base"], t["delta"], w.block_size, w.group_size, w.taps,
                 out=bufs.conv_out, stream=side)
    selector_project(t["h"], t["proj"], w.batch, w.slots, w.top_k, bufs.ws_walk, err=bufs.err,
                     stream=side)
    unary_topk(t["h"], t["lm_head"], w.target_vocab, w.mult, w.cap, w.top_k,
               cand_ids=bufs.cand_ids, cand_u=bufs.cand_u, workspace=bufs.ws_topk, err=bufs.err,
               stream=main)
    if overlap:
        bufs.join.record(side)
        main.wait_event(bufs.join)
    selector_walk_projected(t["A"], t["B"], t["anchors"],
                            bufs.cand_ids.view(w.batch, w.slots, w.top_k),
                            bufs.cand_u.view(w.batch, w.slots, w.top_k), t["temperatures"],
                            t["greedy"], uniforms, w.hidden, bufs.ws_walk, tokens=bufs.tokens,
                            q=bufs.q, err=bufs.err, stream=main)
    d2t_remap(bufs.tokens, t.get("d2t"), w.draft_vocab, w.target_vocab, out=bufs.target_ids,
              err=bufs.err, stream=main)
    return dict(conv_out=bufs.conv_out, cand_ids=bufs.cand_ids, cand_u=bufs.cand_u,
                tokens=bufs.tokens, q=bufs.q, target_ids=bufs.target_ids, err=bufs.err,
                uniforms=uniforms)
