"""Python binding of ``libdq.so``: packed b-bit weight quantization and the
dequantized GEMV / GEMM on MI355X (gfx950).

Two layers, both argument marshalling only (every step runs in the HIP
kernels behind the C ABI declared in ``include/dq.h``):

* ``dq_packed_row_bytes``, ``dq_quantize_pack``, ``dq_row_sumsq``,
  ``dq_quantize_pack_sumsq``, ``dq_unpack``, ``dq_gemv``, ``dq_gemv_batched``, ``dq_gemm``,
  ``dq_stream_read``,
  ``dq_sensitivity``, ``dq_allocate_bits`` -- the C entry points under their
  own names, taking integer addresses (device memory, host memory for the last
  two) and sizes; they return the ``dq_status`` code.
* ``quantize_pack``, ``row_sumsq``, ``quantize_pack_sumsq``, ``unpack``, ``gemv``,
  ``gemv_batched``, ``gemm``, ``stream_read`` -- the same calls on torch tensors (torch provides device
  memory and the current stream); they check device, dtype and contiguity,
  allocate outputs with torch and raise ``DQError`` on a non-zero status.
* ``quantize_pack_asym``, ``unpack_asym``, ``gemv_asym``, ``gemm_asym`` --
  the asymmetric (zero-point) variant on torch tensors.
* ``quantize_pack_group``, ``unpack_group``, ``gemv_group``, ``gemm_group``
  -- group-wise scales (one per g codes of a row) on torch tensors.
* ``quantize_tokens``, ``gemv_i8``, ``gemm_i8`` -- int8 activations (one scale
  per token) and their integer products with packed weights of at most 8 bits.
* ``Cache4``, ``cache4_append``, ``cache4_read``, ``cache4_attention`` -- a paged
  key/value cache held in 4 bits: fill it, read it back, attend over it.
* ``Rope``, ``rotate`` -- rotary positions (halves or neighbours, part of a head, scaled for long
  contexts); ``cache4_append(..., rope=)`` rotates keys on their way into the cache.
* ``draft_tree``, ``cache4_tree_attention``, ``verify_drafts``, ``cache4_keep`` -- a step of drafted
  tokens: the masks of a tree of them, its attention over the cache, their verification
  against the target's probabilities, and the accepted ones' entries moved together.
* ``sensitivity``, ``allocate_bits`` -- the host-side allocation calls on
  numpy arrays (the recipe: one bit width per matrix).
* ``write_packed_file``, ``PackedFile`` -- the on-disk packed-weight format
  (``dq_file_*``): write a recipe's packed matrices from host arrays, map a
  file, read its entries as numpy views and copy them into GPU tensors.

``dq_stream_read`` is not a step of the method: a plain streaming read that
measures what a kernel bound by HBM reaches at a given size.

There is no fallback: if the library is missing or the device is not a GPU,
the calls fail.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "DQError", "DQ_F32", "DQ_BF16", "library_path", "dq_packed_row_bytes", "dq_quantize_pack",
    "dq_unpack", "dq_gemv", "dq_gemm", "dq_stream_read", "dq_status_string", "dq_last_error",
    "packed_row_bytes", "quantize_pack", "unpack", "gemv", "gemm", "stream_read", "load",
    "dq_row_sumsq", "row_sumsq", "dq_quantize_pack_sumsq", "dq_sensitivity", "dq_allocate_bits", "quantize_pack_sumsq",
    "sensitivity", "allocate_bits", "NATIVE_LEVELS", "FULL_LEVELS", "DQFileMatrix",
    "write_packed_file", "PackedFile", "dq_quantize_pack_asym", "dq_unpack_asym",
    "dq_gemv_asym", "dq_gemm_asym", "quantize_pack_asym", "unpack_asym", "gemv_asym",
    "gemm_asym", "dq_quantize_pack_group", "dq_unpack_group", "dq_gemv_group", "dq_gemm_group",
    "quantize_pack_group", "unpack_group", "gemv_group", "gemm_group", "DQGemvItem",
    "GEMV_BATCH_MAX", "dq_gemv_batched", "gemv_batched", "dq_token_row_bytes",
    "dq_quantize_tokens", "dq_gemv_i8", "dq_gemm_i8", "quantize_tokens", "gemv_i8", "gemm_i8",
    "DQCache4", "DQCache4Batch", "dq_cache4_append", "dq_cache4_read",
    "dq_cache4_attention_workspace", "dq_cache4_attention", "Cache4", "cache4_append",
    "cache4_read", "cache4_attention", "DQRope", "dq_rotate", "dq_cache4_append_rope", "dq_draft_tree",
    "dq_cache4_tree_attention_workspace", "dq_cache4_tree_attention", "dq_verify_drafts_workspace",
    "dq_verify_drafts", "dq_cache4_keep", "Rope", "rotate", "draft_tree", "cache4_tree_attention",
    "verify_drafts", "cache4_keep",
]

(DQ_OK, DQ_ERR_NULL, DQ_ERR_BITS, DQ_ERR_SHAPE, DQ_ERR_ALIGN, DQ_ERR_DTYPE, DQ_ERR_HIP,
 DQ_ERR_BUDGET, DQ_ERR_VALUE, DQ_ERR_IO, DQ_ERR_FORMAT) = range(11)
DQ_F32, DQ_BF16 = 0, 1
GEMV_MAX_M = 16
NATIVE_LEVELS = (4, 8, 16)        # hardware-native allocation levels (16 = BF16 kept)
FULL_LEVELS = tuple(range(4, 17))  # every width from 4 to 16

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libdq.so")
_lib = None


class DQFileMatrix(ctypes.Structure):
    """``dq_file_matrix`` of include/dq.h."""
    _fields_ = [("name", ctypes.c_char * 64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("bits", ctypes.c_int32), ("data", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class DQGemvItem(ctypes.Structure):
    """``dq_gemv_item`` of include/dq.h (device addresses and sizes)."""
    _fields_ = [("x", ctypes.c_void_p), ("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("bits", ctypes.c_int32), ("group", ctypes.c_int32), ("zeros", ctypes.c_void_p)]


GEMV_BATCH_MAX = 32
MAX_K_I8 = 65536


class DQCache4(ctypes.Structure):
    """``dq_cache4`` of include/dq.h."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("group", ctypes.c_int32)]


class DQCache4Batch(ctypes.Structure):
    """``dq_cache4_batch`` of include/dq.h."""
    _fields_ = [("starts", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_width", ctypes.c_int64), ("count", ctypes.c_int64)]


class DQRope(ctypes.Structure):
    """``dq_rope`` of include/dq.h."""
    _fields_ = [("turns", ctypes.c_void_p), ("dims", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("factor", ctypes.c_double)]


class DQError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = "%s: %s" % (where, dq_status_string(status))
        if status == DQ_ERR_HIP:
            msg += " (%s)" % dq_last_error()
        super().__init__(msg)
        self.status = status


def load():
    """Load libdq.so (built in-tree by ``mixed_precision_weight_dq_amd.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise ImportError("libdq.so is not built (%s); run __graft_entry__.build() or "
                          "python -m mixed_precision_weight_dq_amd.build" % library_path)
    lib = ctypes.CDLL(library_path)
    i64, i32, vp, st = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32
    lib.dq_packed_row_bytes.argtypes = [i64, i32]
    lib.dq_packed_row_bytes.restype = ctypes.c_size_t
    lib.dq_quantize_pack.argtypes = [vp, i32, i64, i64, i32, vp, vp, vp, vp]
    lib.dq_quantize_pack.restype = st
    lib.dq_unpack.argtypes = [vp, vp, i64, i64, i32, vp, vp, vp]
    lib.dq_unpack.restype = st
    lib.dq_gemv.argtypes = [vp, i64, vp, vp, i64, i64, i32, vp, vp]
    lib.dq_gemv.restype = st
    lib.dq_gemm.argtypes = [vp, i64, vp, vp, i64, i64, i32, vp, vp]
    lib.dq_gemm.restype = st
    lib.dq_gemv_batched.argtypes = [vp, i32, i64, vp]
    lib.dq_gemv_batched.restype = st
    lib.dq_stream_read.argtypes = [vp, i64, vp, i64, vp]
    lib.dq_stream_read.restype = st
    lib.dq_row_sumsq.argtypes = [vp, i32, i64, i64, vp, vp, vp]
    lib.dq_row_sumsq.restype = st
    lib.dq_quantize_pack_asym.argtypes = [vp, i32, i64, i64, i32, vp, vp, vp, vp]
    lib.dq_quantize_pack_asym.restype = st
    lib.dq_unpack_asym.argtypes = [vp, vp, vp, i64, i64, i32, vp, vp, vp]
    lib.dq_unpack_asym.restype = st
    lib.dq_gemv_asym.argtypes = [vp, i64, vp, vp, vp, i64, i64, i32, vp, vp]
    lib.dq_gemv_asym.restype = st
    lib.dq_gemm_asym.argtypes = [vp, i64, vp, vp, vp, i64, i64, i32, vp, vp]
    lib.dq_gemm_asym.restype = st
    lib.dq_quantize_pack_group.argtypes = [vp, i32, i64, i64, i32, i64, vp, vp, vp]
    lib.dq_quantize_pack_group.restype = st
    lib.dq_unpack_group.argtypes = [vp, vp, i64, i64, i32, i64, vp, vp, vp]
    lib.dq_unpack_group.restype = st
    lib.dq_gemv_group.argtypes = [vp, i64, vp, vp, i64, i64, i32, i64, vp, vp]
    lib.dq_gemv_group.restype = st
    lib.dq_gemm_group.argtypes = [vp, i64, vp, vp, i64, i64, i32, i64, vp, vp]
    lib.dq_gemm_group.restype = st
    lib.dq_token_row_bytes.argtypes = [i64]
    lib.dq_token_row_bytes.restype = ctypes.c_size_t
    lib.dq_quantize_tokens.argtypes = [vp, i32, i64, i64, vp, vp, vp, vp]
    lib.dq_quantize_tokens.restype = st
    for fn in (lib.dq_gemv_i8, lib.dq_gemm_i8):
        fn.argtypes = [vp, vp, vp, i64, vp, vp, vp, i64, i64, i32, vp, i32, vp]
        fn.restype = st
    c4, c4b = ctypes.POINTER(DQCache4), ctypes.POINTER(DQCache4Batch)
    lib.dq_cache4_append.argtypes = [c4, c4b, vp, vp, i32, i64, i64, i64, vp]
    lib.dq_cache4_append.restype = st
    lib.dq_cache4_read.argtypes = [c4, c4b, vp, vp, i32, i64, vp]
    lib.dq_cache4_read.restype = st
    lib.dq_cache4_attention_workspace.argtypes = [c4, i64, i64, i32, i64, i64]
    lib.dq_cache4_attention_workspace.restype = ctypes.c_size_t
    lib.dq_cache4_attention.argtypes = [c4, c4b, vp, i64, i64, i32, ctypes.c_float, i64, i64, vp,
                                        vp, ctypes.c_size_t, vp]
    lib.dq_cache4_attention.restype = st
    rp, sz = ctypes.POINTER(DQRope), ctypes.c_size_t
    lib.dq_rotate.argtypes = [rp, vp, i32, i64, i32, i32, i64, i64, vp, vp, i64, i64, vp]
    lib.dq_rotate.restype = st
    lib.dq_cache4_append_rope.argtypes = [c4, c4b, vp, vp, i32, i64, i64, i64, rp, vp, vp]
    lib.dq_cache4_append_rope.restype = st
    lib.dq_draft_tree.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, vp]
    lib.dq_draft_tree.restype = st
    lib.dq_cache4_tree_attention_workspace.argtypes = [c4, i64, i64, i32, i64, i64]
    lib.dq_cache4_tree_attention_workspace.restype = sz
    lib.dq_cache4_tree_attention.argtypes = [c4, c4b, vp, i64, i64, i32, vp, i64, ctypes.c_float, i64, i64,
                                             vp, vp, sz, vp]
    lib.dq_cache4_tree_attention.restype = st
    lib.dq_verify_drafts_workspace.argtypes = [i64, i64]
    lib.dq_verify_drafts_workspace.restype = sz
    lib.dq_verify_drafts.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp, i64, i64, i64, vp, vp, vp, vp, sz, vp]
    lib.dq_verify_drafts.restype = st
    lib.dq_cache4_keep.argtypes = [c4, c4b, vp, vp, i64, vp]
    lib.dq_cache4_keep.restype = st
    fp = ctypes.POINTER(DQFileMatrix)
    lib.dq_file_write.argtypes = [ctypes.c_char_p, fp, i64]
    lib.dq_file_write.restype = st
    lib.dq_file_open.argtypes = [ctypes.c_char_p, ctypes.POINTER(vp)]
    lib.dq_file_open.restype = st
    lib.dq_file_count.argtypes = [vp]
    lib.dq_file_count.restype = i64
    lib.dq_file_matrix_info.argtypes = [vp, i64, fp]
    lib.dq_file_matrix_info.restype = st
    lib.dq_file_verify.argtypes = [vp, i64]
    lib.dq_file_verify.restype = st
    lib.dq_file_load.argtypes = [vp, i64, vp, vp, vp]
    lib.dq_file_load.restype = st
    lib.dq_file_close.argtypes = [vp]
    lib.dq_file_close.restype = None
    lib.dq_quantize_pack_sumsq.argtypes = [vp, i32, i64, i64, i32, vp, vp, vp, vp, vp]
    lib.dq_quantize_pack_sumsq.restype = st
    lib.dq_sensitivity.argtypes = [vp, vp, vp, i64, vp]
    lib.dq_sensitivity.restype = st
    lib.dq_allocate_bits.argtypes = [vp, vp, i64, vp, i32, i64, vp, vp, vp, i64, vp, vp]
    lib.dq_allocate_bits.restype = st
    lib.dq_status_string.argtypes = [st]
    lib.dq_status_string.restype = ctypes.c_char_p
    lib.dq_last_error.argtypes = []
    lib.dq_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


# ---------------------------------------------------------------- raw C ABI

def dq_packed_row_bytes(K: int, bits: int) -> int:
    return int(load().dq_packed_row_bytes(K, bits))


def dq_quantize_pack(w: int, w_dtype: int, N: int, K: int, bits: int, packed: int, scales: int,
                     nonfinite_rows: int = 0, stream: int = 0) -> int:
    return int(load().dq_quantize_pack(w, w_dtype, N, K, bits, packed, scales, nonfinite_rows,
                                       stream))


def dq_quantize_pack_asym(w: int, w_dtype: int, N: int, K: int, bits: int, packed: int,
                          scales: int, zeros: int, stream: int = 0) -> int:
    return int(load().dq_quantize_pack_asym(w, w_dtype, N, K, bits, packed, scales, zeros, stream))


def dq_unpack_asym(packed: int, scales: int, zeros: int, N: int, K: int, bits: int, q_out: int,
                   w_out: int, stream: int = 0) -> int:
    return int(load().dq_unpack_asym(packed, scales, zeros, N, K, bits, q_out, w_out, stream))


def dq_gemv_asym(x: int, M: int, packed: int, scales: int, zeros: int, N: int, K: int,
                 bits: int, y: int, stream: int = 0) -> int:
    return int(load().dq_gemv_asym(x, M, packed, scales, zeros, N, K, bits, y, stream))


def dq_gemm_asym(x: int, M: int, packed: int, scales: int, zeros: int, N: int, K: int,
                 bits: int, y: int, stream: int = 0) -> int:
    return int(load().dq_gemm_asym(x, M, packed, scales, zeros, N, K, bits, y, stream))


def dq_quantize_pack_group(w: int, w_dtype: int, N: int, K: int, bits: int, group: int,
                           packed: int, scales: int, stream: int = 0) -> int:
    return int(load().dq_quantize_pack_group(w, w_dtype, N, K, bits, group, packed, scales, stream))


def dq_unpack_group(packed: int, scales: int, N: int, K: int, bits: int, group: int, q_out: int,
                    w_out: int, stream: int = 0) -> int:
    return int(load().dq_unpack_group(packed, scales, N, K, bits, group, q_out, w_out, stream))


def dq_gemv_group(x: int, M: int, packed: int, scales: int, N: int, K: int, bits: int, group: int,
                  y: int, stream: int = 0) -> int:
    return int(load().dq_gemv_group(x, M, packed, scales, N, K, bits, group, y, stream))


def dq_gemm_group(x: int, M: int, packed: int, scales: int, N: int, K: int, bits: int, group: int,
                  y: int, stream: int = 0) -> int:
    return int(load().dq_gemm_group(x, M, packed, scales, N, K, bits, group, y, stream))


def dq_row_sumsq(w: int, w_dtype: int, N: int, K: int, row_sumsq: int, matrix_sumsq: int,
                 stream: int = 0) -> int:
    return int(load().dq_row_sumsq(w, w_dtype, N, K, row_sumsq, matrix_sumsq, stream))


def dq_quantize_pack_sumsq(w: int, w_dtype: int, N: int, K: int, bits: int, packed: int,
                           scales: int, row_sumsq: int, matrix_sumsq: int, stream: int = 0) -> int:
    return int(load().dq_quantize_pack_sumsq(w, w_dtype, N, K, bits, packed, scales, row_sumsq,
                                             matrix_sumsq, stream))


def dq_sensitivity(h_trace: int, sumsq: int, params: int, n: int, out: int) -> int:
    return int(load().dq_sensitivity(h_trace, sumsq, params, n, out))


def dq_allocate_bits(sensitivity: int, params: int, n: int, levels: int, n_levels: int,
                     budget_bits: int, bits_out: int, step_matrix: int, step_bits: int,
                     step_capacity: int, n_steps: int, loss: int) -> int:
    return int(load().dq_allocate_bits(sensitivity, params, n, levels, n_levels, budget_bits,
                                       bits_out, step_matrix, step_bits, step_capacity, n_steps,
                                       loss))


def dq_unpack(packed: int, scales: int, N: int, K: int, bits: int, q_out: int, w_out: int,
              stream: int = 0) -> int:
    return int(load().dq_unpack(packed, scales, N, K, bits, q_out, w_out, stream))


def dq_gemv(x: int, M: int, packed: int, scales: int, N: int, K: int, bits: int, y: int,
            stream: int = 0) -> int:
    return int(load().dq_gemv(x, M, packed, scales, N, K, bits, y, stream))


def dq_gemv_batched(items: int, count: int, M: int, stream: int = 0) -> int:
    """items: address of a host array of ``DQGemvItem``."""
    return int(load().dq_gemv_batched(items, count, M, stream))


def dq_gemm(x: int, M: int, packed: int, scales: int, N: int, K: int, bits: int, y: int,
            stream: int = 0) -> int:
    return int(load().dq_gemm(x, M, packed, scales, N, K, bits, y, stream))


def dq_token_row_bytes(K: int) -> int:
    return int(load().dq_token_row_bytes(K))


def dq_quantize_tokens(x: int, x_dtype: int, M: int, K: int, codes: int, scales: int, sums: int,
                       stream: int = 0) -> int:
    return int(load().dq_quantize_tokens(x, x_dtype, M, K, codes, scales, sums, stream))


def dq_gemv_i8(x: int, x_scales: int, x_sums: int, M: int, packed: int, scales: int, zeros: int,
               N: int, K: int, bits: int, y: int, y_dtype: int, stream: int = 0) -> int:
    return int(load().dq_gemv_i8(x, x_scales, x_sums, M, packed, scales, zeros, N, K, bits, y,
                                 y_dtype, stream))


def dq_gemm_i8(x: int, x_scales: int, x_sums: int, M: int, packed: int, scales: int, zeros: int,
               N: int, K: int, bits: int, y: int, y_dtype: int, stream: int = 0) -> int:
    return int(load().dq_gemm_i8(x, x_scales, x_sums, M, packed, scales, zeros, N, K, bits, y,
                                 y_dtype, stream))


def dq_cache4_append(cache: DQCache4, batch: DQCache4Batch, k: int, v: int, dtype: int,
                     tokens: int, k_stride: int, v_stride: int, stream: int = 0) -> int:
    return int(load().dq_cache4_append(cache, batch, k, v, dtype, tokens, k_stride, v_stride, stream))


def dq_cache4_read(cache: DQCache4, batch: DQCache4Batch, k: int, v: int, dtype: int, tokens: int,
                   stream: int = 0) -> int:
    return int(load().dq_cache4_read(cache, batch, k, v, dtype, tokens, stream))


def dq_cache4_attention_workspace(cache: DQCache4, count: int, tokens: int, q_heads: int,
                                  max_q: int, max_len: int) -> int:
    return int(load().dq_cache4_attention_workspace(cache, count, tokens, q_heads, max_q, max_len))


def dq_cache4_attention(cache: DQCache4, batch: DQCache4Batch, q: int, tokens: int, q_stride: int,
                        q_heads: int, scale: float, max_q: int, max_len: int, out: int,
                        workspace: int, workspace_bytes: int, stream: int = 0) -> int:
    return int(load().dq_cache4_attention(cache, batch, q, tokens, q_stride, q_heads, scale, max_q,
                                          max_len, out, workspace, workspace_bytes, stream))


def dq_rotate(rope: DQRope, x: int, dtype: int, tokens: int, heads: int, head_dim: int,
              x_token_stride: int, x_head_stride: int, positions: int, out: int,
              out_token_stride: int, out_head_stride: int, stream: int = 0) -> int:
    return int(load().dq_rotate(rope, x, dtype, tokens, heads, head_dim, x_token_stride, x_head_stride,
                                positions, out, out_token_stride, out_head_stride, stream))


def dq_cache4_append_rope(cache: DQCache4, batch: DQCache4Batch, k: int, v: int, dtype: int,
                          tokens: int, k_stride: int, v_stride: int, rope: DQRope, positions: int,
                          stream: int = 0) -> int:
    return int(load().dq_cache4_append_rope(cache, batch, k, v, dtype, tokens, k_stride, v_stride, rope,
                                            positions, stream))


def dq_draft_tree(parents: int, starts: int, lens: int, count: int, tokens: int, words: int, mask: int,
                  positions: int, stream: int = 0) -> int:
    return int(load().dq_draft_tree(parents, starts, lens, count, tokens, words, mask, positions, stream))


def dq_cache4_tree_attention_workspace(cache: DQCache4, count: int, tokens: int, q_heads: int,
                                       max_q: int, max_len: int) -> int:
    return int(load().dq_cache4_tree_attention_workspace(cache, count, tokens, q_heads, max_q, max_len))


def dq_cache4_tree_attention(cache: DQCache4, batch: DQCache4Batch, q: int, tokens: int, q_stride: int,
                             q_heads: int, mask: int, mask_words: int, scale: float, max_q: int,
                             max_len: int, out: int, workspace: int, workspace_bytes: int,
                             stream: int = 0) -> int:
    return int(load().dq_cache4_tree_attention(cache, batch, q, tokens, q_stride, q_heads, mask,
                                               mask_words, scale, max_q, max_len, out, workspace,
                                               workspace_bytes, stream))


def dq_verify_drafts_workspace(count: int, vocab: int) -> int:
    return int(load().dq_verify_drafts_workspace(count, vocab))


def dq_verify_drafts(probs: int, probs_stride: int, draft_probs: int, draft_stride: int, ids: int,
                     parents: int, starts: int, uniforms: int, tokens: int, count: int, vocab: int,
                     path: int, accepted: int, next: int, workspace: int, workspace_bytes: int,
                     stream: int = 0) -> int:
    return int(load().dq_verify_drafts(probs, probs_stride, draft_probs, draft_stride, ids, parents, starts,
                                       uniforms, tokens, count, vocab, path, accepted, next, workspace,
                                       workspace_bytes, stream))


def dq_cache4_keep(cache: DQCache4, batch: DQCache4Batch, path: int, accepted: int, tokens: int,
                   stream: int = 0) -> int:
    return int(load().dq_cache4_keep(cache, batch, path, accepted, tokens, stream))


def dq_stream_read(buf: int, nbytes: int, partial: int, nparts: int, stream: int = 0) -> int:
    return int(load().dq_stream_read(buf, nbytes, partial, nparts, stream))


def dq_status_string(status: int) -> str:
    return load().dq_status_string(status).decode()


def dq_last_error() -> str:
    return load().dq_last_error().decode()


# ----------------------------------------------------------- torch tensors

def packed_row_bytes(K: int, bits: int) -> int:
    rb = dq_packed_row_bytes(K, bits)
    if rb == 0:
        raise DQError(DQ_ERR_SHAPE if 2 <= bits <= 15 else DQ_ERR_BITS, "packed_row_bytes")
    return rb


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream(t):
    torch = _torch()
    return torch.cuda.current_stream(t.device).cuda_stream


def _need(t, name, dtypes, ndim):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be a GPU tensor (got %s)" % (name, t.device))
    if t.dtype not in dtypes:
        raise TypeError("%s dtype %s not in %s" % (name, t.dtype, dtypes))
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %d-D tensor" % (name, ndim))


def _check(status: int, where: str):
    if status != DQ_OK:
        raise DQError(status, where)


def quantize_pack(w, bits: int, packed=None, scales=None, nonfinite=None):
    """W[N, K] (float32 or bfloat16, on the GPU) -> (packed int32 [N, row_bytes/4] holding
    the uint32 words, scales float32 [N]).  nonfinite: optional int32 [1] tensor
    that receives the number of rows holding a NaN or an infinity."""
    torch = _torch()
    _need(w, "w", (torch.float32, torch.bfloat16), 2)
    N, K = w.shape
    rw = packed_row_bytes(K, bits) // 4
    if packed is None:
        packed = torch.empty((N, rw), dtype=torch.int32, device=w.device)
    if scales is None:
        scales = torch.empty((N,), dtype=torch.float32, device=w.device)
    _need(packed, "packed", (torch.int32,), 2)
    _need(scales, "scales", (torch.float32,), 1)
    if tuple(packed.shape) != (N, rw) or tuple(scales.shape) != (N,):
        raise ValueError("packed/scales shape mismatch")
    if nonfinite is not None:
        _need(nonfinite, "nonfinite", (torch.int32,), 1)
        if nonfinite.shape[0] != 1:
            raise ValueError("nonfinite must be [1]")
    dt = DQ_BF16 if w.dtype == torch.bfloat16 else DQ_F32
    _check(dq_quantize_pack(w.data_ptr(), dt, N, K, bits, packed.data_ptr(), scales.data_ptr(),
                            nonfinite.data_ptr() if nonfinite is not None else 0, _stream(w)),
           "dq_quantize_pack")
    return packed, scales


def quantize_pack_asym(w, bits: int):
    """Asymmetric per-row quantization: W[N, K] (float32 / bfloat16, GPU) ->
    (packed int32 [N, row_words] holding unsigned codes, scales float32 [N],
    zeros int32 [N])."""
    torch = _torch()
    _need(w, "w", (torch.float32, torch.bfloat16), 2)
    N, K = w.shape
    packed = torch.empty((N, packed_row_bytes(K, bits) // 4), dtype=torch.int32, device=w.device)
    scales = torch.empty((N,), dtype=torch.float32, device=w.device)
    zeros = torch.empty((N,), dtype=torch.int32, device=w.device)
    dt = DQ_BF16 if w.dtype == torch.bfloat16 else DQ_F32
    _check(dq_quantize_pack_asym(w.data_ptr(), dt, N, K, bits, packed.data_ptr(), scales.data_ptr(),
                                 zeros.data_ptr(), _stream(w)), "dq_quantize_pack_asym")
    return packed, scales, zeros


def unpack_asym(packed, scales, zeros, K: int, bits: int, want_q: bool = True,
                want_w: bool = False):
    """(q = u - z int32 [N, K] or None, w_hat float32 [N, K] or None)."""
    torch = _torch()
    _need(packed, "packed", (torch.int32,), 2)
    _need(zeros, "zeros", (torch.int32,), 1)
    N = packed.shape[0]
    if packed.shape[1] != packed_row_bytes(K, bits) // 4 or zeros.shape[0] != N:
        raise ValueError("packed / zeros do not match N, K and bits")
    q = torch.empty((N, K), dtype=torch.int32, device=packed.device) if want_q else None
    w = torch.empty((N, K), dtype=torch.float32, device=packed.device) if want_w else None
    if scales is not None:
        _need(scales, "scales", (torch.float32,), 1)
    _check(dq_unpack_asym(packed.data_ptr(), scales.data_ptr() if scales is not None else 0,
                          zeros.data_ptr(), N, K, bits, q.data_ptr() if q is not None else 0,
                          w.data_ptr() if w is not None else 0, _stream(packed)), "dq_unpack_asym")
    return q, w


def _matmul_asym(fn, name, x, packed, scales, zeros, K: int, bits: int, y=None):
    torch = _torch()
    _need(x, "x", (torch.bfloat16,), 2)
    _need(packed, "packed", (torch.int32,), 2)
    _need(scales, "scales", (torch.float32,), 1)
    _need(zeros, "zeros", (torch.int32,), 1)
    M, N = x.shape[0], packed.shape[0]
    if (x.shape[1] != K or packed.shape[1] != packed_row_bytes(K, bits) // 4
            or scales.shape[0] != N or zeros.shape[0] != N):
        raise ValueError("shape mismatch between x, packed, scales, zeros, K and bits")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _need(y, "y", (torch.float32,), 2)
    if tuple(y.shape) != (M, N):
        raise ValueError("y must be [M, N]")
    _check(fn(x.data_ptr(), M, packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(), N, K, bits,
              y.data_ptr(), _stream(x)), name)
    return y


def gemv_asym(x, packed, scales, zeros, K: int, bits: int, y=None):
    """y = s * x . (u - z)^T for 1 <= M <= 16."""
    return _matmul_asym(dq_gemv_asym, "dq_gemv_asym", x, packed, scales, zeros, K, bits, y)


def gemm_asym(x, packed, scales, zeros, K: int, bits: int, y=None):
    """y = s * x . (u - z)^T on the matrix cores (any M >= 1)."""
    return _matmul_asym(dq_gemm_asym, "dq_gemm_asym", x, packed, scales, zeros, K, bits, y)


def quantize_pack_group(w, bits: int, group: int):
    """Group-wise scales: W[N, K] -> (packed int32 [N, row_words], scales float32
    [N, ceil(K / group)])."""
    torch = _torch()
    _need(w, "w", (torch.float32, torch.bfloat16), 2)
    N, K = w.shape
    packed = torch.empty((N, packed_row_bytes(K, bits) // 4), dtype=torch.int32, device=w.device)
    scales = torch.empty((N, -(-K // group)), dtype=torch.float32, device=w.device)
    dt = DQ_BF16 if w.dtype == torch.bfloat16 else DQ_F32
    _check(dq_quantize_pack_group(w.data_ptr(), dt, N, K, bits, group, packed.data_ptr(),
                                  scales.data_ptr(), _stream(w)), "dq_quantize_pack_group")
    return packed, scales


def unpack_group(packed, scales, K: int, bits: int, group: int, want_q: bool = True,
                 want_w: bool = False):
    torch = _torch()
    _need(packed, "packed", (torch.int32,), 2)
    N = packed.shape[0]
    if packed.shape[1] != packed_row_bytes(K, bits) // 4:
        raise ValueError("packed row length does not match K and bits")
    if scales is not None:
        _need(scales, "scales", (torch.float32,), 2)
        if tuple(scales.shape) != (N, -(-K // group)):
            raise ValueError("scales must be [N, ceil(K / group)]")
    q = torch.empty((N, K), dtype=torch.int32, device=packed.device) if want_q else None
    w = torch.empty((N, K), dtype=torch.float32, device=packed.device) if want_w else None
    _check(dq_unpack_group(packed.data_ptr(), scales.data_ptr() if scales is not None else 0, N, K,
                           bits, group, q.data_ptr() if q is not None else 0,
                           w.data_ptr() if w is not None else 0, _stream(packed)),
           "dq_unpack_group")
    return q, w


def _matmul_group(fn, name, x, packed, scales, K: int, bits: int, group: int, y=None):
    torch = _torch()
    _need(x, "x", (torch.bfloat16,), 2)
    _need(packed, "packed", (torch.int32,), 2)
    _need(scales, "scales", (torch.float32,), 2)
    M, N = x.shape[0], packed.shape[0]
    if (x.shape[1] != K or packed.shape[1] != packed_row_bytes(K, bits) // 4
            or tuple(scales.shape) != (N, -(-K // group))):
        raise ValueError("shape mismatch between x, packed, scales, K, bits and group")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _need(y, "y", (torch.float32,), 2)
    if tuple(y.shape) != (M, N):
        raise ValueError("y must be [M, N]")
    _check(fn(x.data_ptr(), M, packed.data_ptr(), scales.data_ptr(), N, K, bits, group,
              y.data_ptr(), _stream(x)), name)
    return y


def gemv_group(x, packed, scales, K: int, bits: int, group: int, y=None):
    """y = sum_k x q s[n, k / group] for 1 <= M <= 16."""
    return _matmul_group(dq_gemv_group, "dq_gemv_group", x, packed, scales, K, bits, group, y)


def gemm_group(x, packed, scales, K: int, bits: int, group: int, y=None):
    """The same on the bf16 matrix cores (any M >= 1)."""
    return _matmul_group(dq_gemm_group, "dq_gemm_group", x, packed, scales, K, bits, group, y)


def row_sumsq(w, want_total: bool = True):
    """fp64 sum of w^2 of every row of W[N, K] (float32 or bfloat16, on the GPU),
    and of the whole matrix.  Returns (row_sumsq float64 [N], matrix_sumsq float64
    [1] or None)."""
    torch = _torch()
    _need(w, "w", (torch.float32, torch.bfloat16), 2)
    N, K = w.shape
    row = torch.empty((N,), dtype=torch.float64, device=w.device)
    total = torch.empty((1,), dtype=torch.float64, device=w.device) if want_total else None
    dt = DQ_BF16 if w.dtype == torch.bfloat16 else DQ_F32
    _check(dq_row_sumsq(w.data_ptr(), dt, N, K, row.data_ptr(),
                        total.data_ptr() if total is not None else 0, _stream(w)), "dq_row_sumsq")
    return row, total


def quantize_pack_sumsq(w, bits: int, want_total: bool = True):
    """``quantize_pack`` plus the fp64 sum of w^2 of every row, taken in the same
    pass.  Returns (packed, scales, row_sumsq float64 [N], matrix_sumsq float64 [1]
    or None)."""
    torch = _torch()
    _need(w, "w", (torch.float32, torch.bfloat16), 2)
    N, K = w.shape
    rw = packed_row_bytes(K, bits) // 4
    packed = torch.empty((N, rw), dtype=torch.int32, device=w.device)
    scales = torch.empty((N,), dtype=torch.float32, device=w.device)
    row = torch.empty((N,), dtype=torch.float64, device=w.device)
    total = torch.empty((1,), dtype=torch.float64, device=w.device) if want_total else None
    dt = DQ_BF16 if w.dtype == torch.bfloat16 else DQ_F32
    _check(dq_quantize_pack_sumsq(w.data_ptr(), dt, N, K, bits, packed.data_ptr(),
                                  scales.data_ptr(), row.data_ptr(),
                                  total.data_ptr() if total is not None else 0, _stream(w)),
           "dq_quantize_pack_sumsq")
    return packed, scales, row, total


def _host(a, dtype, name):
    import numpy as np
    a = np.ascontiguousarray(a, dtype=dtype)
    if a.ndim != 1:
        raise ValueError("%s must be 1-D" % name)
    return a


def _addr(a) -> int:
    return a.ctypes.data


def sensitivity(h_trace, sumsq, params):
    """Sensitivity per matrix, h_trace * (sumsq / params), on the host (numpy in,
    numpy float64 out)."""
    import numpy as np
    h = _host(h_trace, np.float64, "h_trace")
    ss = _host(sumsq, np.float64, "sumsq")
    p = _host(params, np.int64, "params")
    if not h.size == ss.size == p.size:
        raise ValueError("h_trace, sumsq and params must have one entry per matrix")
    out = np.empty(h.size, dtype=np.float64)
    _check(dq_sensitivity(_addr(h), _addr(ss), _addr(p), h.size, _addr(out)), "dq_sensitivity")
    return out


def allocate_bits(sens, params, levels=FULL_LEVELS, budget_bits=None):
    """Water-filling allocation on the host.  Returns (bits int32 [n], steps as a
    list of (matrix, new width) in the order taken, predicted loss).  A budget
    of None walks the whole frontier."""
    import numpy as np
    s = _host(sens, np.float64, "sensitivity")
    p = _host(params, np.int64, "params")
    lv = _host(levels, np.int32, "levels")
    if s.size != p.size:
        raise ValueError("one sensitivity and one parameter count per matrix")
    bits = np.empty(s.size, dtype=np.int32)
    cap = s.size * max(lv.size - 1, 0)
    sm = np.empty(max(cap, 1), dtype=np.int64)
    sb = np.empty(max(cap, 1), dtype=np.int32)
    nsteps = np.zeros(1, dtype=np.int64)
    loss = np.zeros(1, dtype=np.float64)
    budget = -1 if budget_bits is None else int(budget_bits)
    if budget_bits is not None and budget < 0:
        raise ValueError("budget_bits must be >= 0 (None = no limit)")
    _check(dq_allocate_bits(_addr(s), _addr(p), s.size, _addr(lv), lv.size, budget, _addr(bits),
                            _addr(sm), _addr(sb), cap, _addr(nsteps), _addr(loss)),
           "dq_allocate_bits")
    n = int(nsteps[0])
    return bits, list(zip(sm[:n].tolist(), sb[:n].tolist())), float(loss[0])


def unpack(packed, scales, K: int, bits: int, want_q: bool = True, want_w: bool = False):
    """packed [N, row_words] -> (q int32 [N, K] or None, w_hat float32 [N, K] or None)."""
    torch = _torch()
    _need(packed, "packed", (torch.int32,), 2)
    N = packed.shape[0]
    if packed.shape[1] != packed_row_bytes(K, bits) // 4:
        raise ValueError("packed row length does not match K and bits")
    q = torch.empty((N, K), dtype=torch.int32, device=packed.device) if want_q else None
    w = torch.empty((N, K), dtype=torch.float32, device=packed.device) if want_w else None
    if scales is not None:
        _need(scales, "scales", (torch.float32,), 1)
    _check(dq_unpack(packed.data_ptr(), scales.data_ptr() if scales is not None else 0, N, K, bits,
                     q.data_ptr() if q is not None else 0, w.data_ptr() if w is not None else 0,
                     _stream(packed)), "dq_unpack")
    return q, w


def _matmul(fn, name, x, packed, scales, K: int, bits: int, y=None):
    torch = _torch()
    _need(x, "x", (torch.bfloat16,), 2)
    _need(packed, "packed", (torch.int32,), 2)
    _need(scales, "scales", (torch.float32,), 1)
    M = x.shape[0]
    N = packed.shape[0]
    if x.shape[1] != K or packed.shape[1] != packed_row_bytes(K, bits) // 4 or scales.shape[0] != N:
        raise ValueError("shape mismatch between x, packed, scales, K and bits")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _need(y, "y", (torch.float32,), 2)
    if tuple(y.shape) != (M, N):
        raise ValueError("y must be [M, N]")
    _check(fn(x.data_ptr(), M, packed.data_ptr(), scales.data_ptr(), N, K, bits, y.data_ptr(),
              _stream(x)), name)
    return y


def gemv(x, packed, scales, K: int, bits: int, y=None):
    """y[M, N] = x . dequant(W)^T for 1 <= M <= 16 (fp32 accumulate)."""
    return _matmul(dq_gemv, "dq_gemv", x, packed, scales, K, bits, y)


def gemv_batched(items, ys=None):
    """Several decode products in one call: items is a list of (x, packed,
    scales, K, bits), optionally followed by zeros (int32 [N] zero points of
    asymmetric codes, or None) and group (codes per group scale, scales then
    [N, ceil(K / group)]; 0 for a scale per row); bf16 x [M, K] with the same
    M for all; x and weights may be shared between items.  Returns the list of
    y [M, N] (or fills ``ys``).  The items of each scheme that fit one launch
    share it; the others run as one launch each of their scheme's entry point."""
    torch = _torch()
    if not 1 <= len(items) <= GEMV_BATCH_MAX:
        raise ValueError("1 to %d items" % GEMV_BATCH_MAX)
    arr = (DQGemvItem * len(items))()
    out = []
    M = None
    for i, item in enumerate(items):
        if not 5 <= len(item) <= 7:
            raise ValueError("item %d: (x, packed, scales, K, bits[, zeros[, group]])" % i)
        x, packed, scales, K, bits = item[:5]
        zeros = item[5] if len(item) > 5 else None
        group = item[6] if len(item) > 6 else 0
        _need(x, "x", (torch.bfloat16,), 2)
        _need(packed, "packed", (torch.int32,), 2)
        N = packed.shape[0]
        if group:
            _need(scales, "scales", (torch.float32,), 2)
            ok_scales = tuple(scales.shape) == (N, -(-K // group))
        else:
            _need(scales, "scales", (torch.float32,), 1)
            ok_scales = scales.shape[0] == N
        if zeros is not None:
            _need(zeros, "zeros", (torch.int32,), 1)
            ok_scales = ok_scales and zeros.shape[0] == N
        if M is None:
            M = x.shape[0]
        if x.shape[0] != M or x.shape[1] != K or \
                packed.shape[1] != packed_row_bytes(K, bits) // 4 or not ok_scales:
            raise ValueError("item %d: shape mismatch between x, packed, scales, zeros, K and bits" % i)
        y = ys[i] if ys is not None else torch.empty((M, N), dtype=torch.float32, device=x.device)
        _need(y, "y", (torch.float32,), 2)
        if tuple(y.shape) != (M, N):
            raise ValueError("item %d: y must be [M, N]" % i)
        arr[i] = DQGemvItem(x.data_ptr(), packed.data_ptr(), scales.data_ptr(), y.data_ptr(), N, K,
                            bits, group, zeros.data_ptr() if zeros is not None else 0)
        out.append(y)
    _check(dq_gemv_batched(ctypes.addressof(arr), len(items), M, _stream(items[0][0])),
           "dq_gemv_batched")
    return out


def gemm(x, packed, scales, K: int, bits: int, y=None):
    """y[M, N] = x . dequant(W)^T on the bf16 matrix cores (any M >= 1)."""
    return _matmul(dq_gemm, "dq_gemm", x, packed, scales, K, bits, y)


def _dtype_code(dtype, name):
    torch = _torch()
    if dtype is torch.float32:
        return DQ_F32
    if dtype is torch.bfloat16:
        return DQ_BF16
    raise TypeError("%s must be torch.float32 or torch.bfloat16 (got %s)" % (name, dtype))


def _fast_need(t, name, dtype, ndim, dev):
    """``_need`` for one dtype, in a few attribute reads where nothing is wrong (the calls of a
    decode step cost the host more than their kernels take); all tensors on GPU ``dev``."""
    try:
        if (t.is_cuda and t.dtype is dtype and t.dim() == ndim and t.is_contiguous()
                and t.get_device() == dev):
            return
    except AttributeError:
        pass
    _need(t, name, (dtype,), ndim)
    raise ValueError("%s: all tensors must be on one GPU (cuda:%d and %s)" % (name, dev, t.device))


def _gpu_index(t, name):
    try:
        if t.is_cuda:
            return t.get_device()
    except AttributeError:
        raise TypeError("%s must be a torch.Tensor" % name) from None
    raise ValueError("%s must be a GPU tensor (got %s)" % (name, t.device))


def _launch(where, dev, fn, *args):
    """fn(*args, stream) on GPU ``dev`` and its current stream."""
    torch = _torch()
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status != DQ_OK:
        raise DQError(status, where)


def quantize_tokens(x, codes=None, scales=None, sums=None):
    """x[M, K] (float32 or bfloat16, on the GPU) -> (codes int8 [M, K rounded up to 128],
    scales float32 [M], sums int32 [M]): one symmetric int8 scale per token, and each
    token's sum of codes."""
    torch = _torch()
    dev = _gpu_index(x, "x")
    kind = _dtype_code(x.dtype, "x")
    _fast_need(x, "x", x.dtype, 2, dev)
    M, K = x.shape
    if not 1 <= K <= MAX_K_I8:
        raise DQError(DQ_ERR_SHAPE, "quantize_tokens")
    pitch = (K + 127) & -128
    if codes is None:
        codes = x.new_empty((M, pitch), dtype=torch.int8)
    else:
        _fast_need(codes, "codes", torch.int8, 2, dev)
        if tuple(codes.shape) != (M, pitch):
            raise ValueError("codes must be [M, %d]" % pitch)
    if scales is None:
        scales = x.new_empty((M,), dtype=torch.float32)
    else:
        _fast_need(scales, "scales", torch.float32, 1, dev)
    if sums is None:
        sums = x.new_empty((M,), dtype=torch.int32)
    else:
        _fast_need(sums, "sums", torch.int32, 1, dev)
    if scales.shape[0] != M or sums.shape[0] != M:
        raise ValueError("scales and sums must be [M]")
    _launch("dq_quantize_tokens", dev, load().dq_quantize_tokens, x.data_ptr(), kind, M, K,
            codes.data_ptr(), scales.data_ptr(), sums.data_ptr())
    return codes, scales, sums


def _matmul_i8(fn, name, codes, x_scales, x_sums, packed, scales, K, bits, zeros, y, dtype):
    torch = _torch()
    dev = _gpu_index(codes, "codes")
    _fast_need(codes, "codes", torch.int8, 2, dev)
    _fast_need(x_scales, "x_scales", torch.float32, 1, dev)
    _fast_need(x_sums, "x_sums", torch.int32, 1, dev)
    _fast_need(packed, "packed", torch.int32, 2, dev)
    _fast_need(scales, "scales", torch.float32, 1, dev)
    (M, pitch), (N, words) = codes.shape, packed.shape
    if not 2 <= bits <= 8:
        raise DQError(DQ_ERR_BITS, name)
    if not 1 <= K <= MAX_K_I8:
        raise DQError(DQ_ERR_SHAPE, name)
    if (pitch != (K + 127) & -128 or x_scales.shape[0] != M or x_sums.shape[0] != M
            or words != ((K * bits + 7) // 8 + 127) // 128 * 32 or scales.shape[0] != N):
        raise ValueError("shape mismatch between codes, x_scales, x_sums, packed, scales, K and bits")
    if zeros is not None:
        _fast_need(zeros, "zeros", torch.int32, 1, dev)
        if zeros.shape[0] != N:
            raise ValueError("zeros must be [N]")
        zeros = zeros.data_ptr()
    if y is None:
        y = codes.new_empty((M, N), dtype=torch.float32 if dtype is None else dtype)
        kind = _dtype_code(y.dtype, "dtype")
    else:
        kind = _dtype_code(y.dtype, "y")
        if dtype is not None and y.dtype != dtype:
            raise TypeError("y is %s, dtype %s" % (y.dtype, dtype))
        _fast_need(y, "y", y.dtype, 2, dev)
        if tuple(y.shape) != (M, N):
            raise ValueError("y must be [M, N]")
    _launch(name, dev, fn, codes.data_ptr(), x_scales.data_ptr(), x_sums.data_ptr(), M,
            packed.data_ptr(), scales.data_ptr(), zeros, N, K, bits, y.data_ptr(), kind)
    return y


def gemv_i8(codes, x_scales, x_sums, packed, scales, K: int, bits: int, zeros=None, y=None,
            dtype=None):
    """y[M, N] = x_scales * scales * codes . (u - z)^T for 1 <= M <= 16: ``quantize_tokens``'
    outputs times weights from ``quantize_pack`` (or, with ``zeros``, ``quantize_pack_asym``) of
    at most 8 bits; y float32 (the default) or bfloat16."""
    return _matmul_i8(load().dq_gemv_i8, "dq_gemv_i8", codes, x_scales, x_sums, packed, scales, K,
                      bits, zeros, y, dtype)


def gemm_i8(codes, x_scales, x_sums, packed, scales, K: int, bits: int, zeros=None, y=None,
            dtype=None):
    """The same for any M >= 1."""
    return _matmul_i8(load().dq_gemm_i8, "dq_gemm_i8", codes, x_scales, x_sums, packed, scales, K,
                      bits, zeros, y, dtype)


class Cache4:
    """A paged key/value cache in 4 bits: k_codes, v_codes int32 [pages, kv_heads, P, D / 8]
    and k_scales, v_scales float32 [pages, kv_heads, D / g, P], contiguous GPU tensors that
    the caller owns (``Cache4.empty`` allocates them).  Its attributes cannot be set: other
    tensors, a larger cache for instance, make another ``Cache4``, and a call on one whose
    tensors were moved in place is refused.  The sequences of a call are given by
    ``starts`` int32 [count + 1] (token rows of each sequence), ``lens`` int32 [count] (cached
    tokens, the call's own included) and ``table`` int32 [count, width] (pages)."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        torch = _torch()
        dev = _gpu_index(k_codes, "k_codes")
        for t, name in ((k_codes, "k_codes"), (v_codes, "v_codes")):
            _fast_need(t, name, torch.int32, 4, dev)
        for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            _fast_need(t, name, torch.float32, 4, dev)
        pages, heads, P, words = k_codes.shape
        groups = k_scales.shape[2]
        if (v_codes.shape != k_codes.shape or v_scales.shape != k_scales.shape
                or tuple(k_scales.shape) != (pages, heads, groups, P)
                or groups < 1 or words * 8 % groups):
            raise ValueError("codes must be [pages, kv_heads, P, D / 8], scales [pages, kv_heads, D / g, P]")
        at = tuple(t.data_ptr() for t in (k_codes, v_codes, k_scales, v_scales))
        D, g = words * 8, words * 8 // groups
        self.__dict__.update(
            k_codes=k_codes, v_codes=v_codes, k_scales=k_scales, v_scales=v_scales, pages=pages,
            kv_heads=heads, page_size=P, head_dim=D, group=g, device_index=dev, _at=at,
            _c=DQCache4(*at, pages, heads, D, P, g))

    def __setattr__(self, name, value):
        raise AttributeError("a Cache4's attributes are fixed: make another one (%s)" % name)

    def __delattr__(self, name):
        self.__setattr__(name, None)

    def _struct(self):
        """The C struct, if the tensors still lie where it says."""
        if (self.k_codes.data_ptr(), self.v_codes.data_ptr(), self.k_scales.data_ptr(),
                self.v_scales.data_ptr()) != self._at:
            raise ValueError("the cache's tensors were moved: make another Cache4 of them")
        return self._c

    @classmethod
    def empty(cls, pages: int, kv_heads: int, head_dim: int, page_size: int = 64, group: int = 32,
              device="cuda"):
        torch = _torch()
        if (head_dim not in (64, 128, 256) or group not in (32, 64, 128) or group > head_dim
                or not 16 <= page_size <= 256 or page_size & (page_size - 1)):
            raise DQError(DQ_ERR_SHAPE, "Cache4.empty")
        codes = (pages, kv_heads, page_size, head_dim // 8)
        scales = (pages, kv_heads, head_dim // group, page_size)
        return cls(*(torch.zeros(codes, dtype=torch.int32, device=device) for _ in range(2)),
                   *(torch.zeros(scales, dtype=torch.float32, device=device) for _ in range(2)))

    @property
    def tensors(self):
        return self.k_codes, self.v_codes, self.k_scales, self.v_scales


def _batch4(starts, lens, table, dev):
    torch = _torch()
    _fast_need(starts, "starts", torch.int32, 1, dev)
    _fast_need(lens, "lens", torch.int32, 1, dev)
    _fast_need(table, "table", torch.int32, 2, dev)
    count = lens.shape[0]
    rows, width = table.shape
    if starts.shape[0] != count + 1 or rows != count:
        raise ValueError("starts must be [count + 1], lens [count], table [count, width]")
    return DQCache4Batch(starts.data_ptr(), lens.data_ptr(), table.data_ptr(), width, count)


def _token_rows(t, name, heads, D, dev):
    """Checks t [tokens, heads, D] with contiguous heads on GPU ``dev``; returns its token stride."""
    if _gpu_index(t, name) != dev:
        raise ValueError("%s: all tensors must be on one GPU (cuda:%d and %s)" % (name, dev, t.device))
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != D:
        raise ValueError("%s must be [tokens, %d, %d]" % (name, heads, D))
    token, head, dim = t.stride()
    if dim != 1 or (heads > 1 and head != D):
        raise ValueError("%s: the heads of a token must be contiguous" % name)
    return token if shape[0] > 1 else heads * D


class Rope:
    """Rotary positions: pairs of a head's first ``dims`` dimensions, (i, i + dims / 2) or,
    ``interleaved``, (2 i, 2 i + 1), turn by ``base ** (-2 i / dims)`` radians a position.

    ``scaling`` stretches them for contexts longer than those of training, by ``factor`` s > 0:
    ``dict(kind="linear", factor=s)``, every frequency divided by s;
    ``dict(kind="ntk", factor=s)``, base times s ** (dims / (dims - 2));
    ``dict(kind="yarn", factor=s, length=L, fast=32, slow=1)``, a ramp over the pairs from the one that
    turns ``fast`` times over the trained length L (as it was) to the one that turns ``slow`` times
    (divided by s), and vectors times 0.1 ln s + 1 (``amplitude=`` sets another factor);
    ``dict(kind="bands", factor=s, length=L, low=1, high=4)``, wavelengths below L / high as they were, above
    L / low divided by s, between them mixed;
    ``dict(kind="list", divisors=[...], amplitude=1.0)``, a divisor for each pair.
    Attributes (fixed): turns (float64 GPU tensor [dims / 2], turns a position), dims, interleaved,
    factor (of the rotated vector)."""

    def __init__(self, dims: int, base: float = 10000.0, interleaved: bool = False, scaling=None,
                 device="cuda"):
        torch = _torch()
        turns, factor = _rope_turns(dims, base, scaling)
        turns = torch.tensor(turns, dtype=torch.float64).to(device)
        dev = _gpu_index(turns, "device")
        self.__dict__.update(turns=turns, dims=dims, interleaved=bool(interleaved), factor=factor,
                             device_index=dev, _at=turns.data_ptr(),
                             _c=DQRope(turns.data_ptr(), dims, bool(interleaved), factor))

    def __setattr__(self, name, value):
        raise AttributeError("a Rope's attributes are fixed: make another one (%s)" % name)

    def __delattr__(self, name):
        self.__setattr__(name, None)

    def _struct(self, dev):
        """The C struct, for a call on GPU ``dev``."""
        if dev != self.device_index:
            raise ValueError("the rope is on cuda:%d, the call on cuda:%d" % (self.device_index, dev))
        if self.turns.data_ptr() != self._at:
            raise ValueError("the rope's tensor was moved: make another Rope")
        return self._c


def _rope_turns(dims, base, scaling):
    """(turns a position of each pair, factor of the rotated vector), on the host in float64."""
    import math
    if not 2 <= dims <= 4096 or dims % 2:
        raise DQError(DQ_ERR_SHAPE, "Rope")
    if not (math.isfinite(base) and base > 1):
        raise ValueError("base must be finite and above 1")
    given = dict(scaling or {})
    kind = given.pop("kind", None)
    allowed = {None: (), "linear": ("factor",), "ntk": ("factor",),
               "yarn": ("factor", "length", "fast", "slow", "amplitude"),
               "bands": ("factor", "length", "low", "high"), "list": ("divisors", "amplitude")}
    if kind not in allowed:
        raise ValueError("scaling kind must be linear, ntk, yarn, bands or list (got %r)" % (kind,))
    if kind in ("linear", "ntk"):
        given = {k: v for k, v in given.items() if k != "length"}  # (they need none)
    unknown = set(given) - set(allowed[kind])
    if unknown:
        raise ValueError("scaling %s does not take %s" % (kind, ", ".join(sorted(map(str, unknown)))))

    def number(name, default=None):
        value = given.get(name, default)
        if isinstance(value, bool) or not isinstance(value, (int, float)) or not math.isfinite(value) or value <= 0:
            raise ValueError("scaling %s: %s must be a positive number (got %r)" % (kind, name, value))
        return float(value)

    pairs = range(dims // 2)
    factor = 1.0
    s = number("factor") if "factor" in allowed[kind] else 1.0
    if kind == "ntk":
        if dims == 2:
            raise ValueError("scaling ntk needs more than one pair")
        base = base * s ** (dims / (dims - 2))
    rate = [base ** (-2 * i / dims) for i in pairs]
    if kind == "linear":
        rate = [r / s for r in rate]
    elif kind == "yarn":
        length, fast, slow = number("length"), number("fast", 32), number("slow", 1)
        if fast < slow:
            raise ValueError("scaling yarn: fast must be at least slow")
        # the pair that turns n times over the length
        at = [dims * math.log(length / (2 * math.pi * n)) / (2 * math.log(base)) for n in (fast, slow)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), dims - 1)
        ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in pairs]
        rate = [r / s * w + r * (1 - w) for r, w in zip(rate, ramp)]
        factor = number("amplitude", 0.1 * math.log(s) + 1 if s > 1 else 1.0)
    elif kind == "bands":
        length, low, high = number("length"), number("low", 1), number("high", 4)
        if high <= low:
            raise ValueError("scaling bands: high must be above low")
        mix = [min(max((length * r / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for r in rate]
        rate = [r / s * (1 - w) + r * w for r, w in zip(rate, mix)]
    elif kind == "list":
        divisors = [float(d) for d in given.get("divisors", ())]
        if len(divisors) != dims // 2 or not all(math.isfinite(d) and d > 0 for d in divisors):
            raise ValueError("scaling list: divisors must be dims / 2 positive numbers")
        rate = [r / d for r, d in zip(rate, divisors)]
        factor = number("amplitude", 1.0)
    return [r / (2 * math.pi) for r in rate], factor


def _head_rows(t, name, shape, dev):
    """Checks t [tokens, heads, D] with contiguous dimensions on GPU ``dev``; returns its token and
    head strides."""
    if _gpu_index(t, name) != dev:
        raise ValueError("%s: all tensors must be on one GPU (cuda:%d and %s)" % (name, dev, t.device))
    if t.dim() != 3 or (shape is not None and t.shape != shape):
        raise ValueError("%s must be [tokens, heads, D]" % name)
    tokens, heads, D = t.shape
    token, head, dim = t.stride()
    if dim != 1 and D > 1:
        raise ValueError("%s: a head's dimensions must be contiguous" % name)
    if heads == 1:
        head = D
    if tokens == 1:
        token = heads * head
    return token, head


def _positions(positions, tokens, dev):
    torch = _torch()
    _fast_need(positions, "positions", torch.int32, 1, dev)
    if positions.shape[0] != tokens:
        raise ValueError("positions must be [tokens]")
    return positions.data_ptr()


def rotate(rope: Rope, x, positions, out=None):
    """x [tokens, heads, D] (float32 or bfloat16; tokens and heads may be strided) with its first
    ``rope.dims`` dimensions rotated at positions int32 [tokens].  out: a tensor of x's shape
    and type, x itself among them (a new contiguous one unless given)."""
    dev = _gpu_index(x, "x")
    kind = _dtype_code(x.dtype, "x")
    token, head = _head_rows(x, "x", None, dev)
    tokens, heads, D = x.shape
    at = _positions(positions, tokens, dev)
    if out is None:
        out = x.new_empty((tokens, heads, D))
        out_token, out_head = heads * D, D
    else:
        out_token, out_head = _head_rows(out, "out", x.shape, dev)
        if out.dtype != x.dtype:
            raise ValueError("out must have x's type")
    _launch("dq_rotate", dev, load().dq_rotate, rope._struct(dev), x.data_ptr(), kind, tokens, heads, D,
            token, head, at, out.data_ptr(), out_token, out_head)
    return out


def cache4_append(cache: Cache4, k, v, starts, lens, table, rope=None, positions=None) -> None:
    """Quantize k, v [tokens, kv_heads, D] (float32 or bfloat16; tokens may be strided) into
    the pages of their positions.  rope: a ``Rope`` (dims a multiple of 16, at most D) that
    rotates the keys on the way, at ``positions`` int32 [tokens] or, without them, at each token's
    position in its sequence."""
    dev = cache.device_index
    ks = _token_rows(k, "k", cache.kv_heads, cache.head_dim, dev)
    vs = _token_rows(v, "v", cache.kv_heads, cache.head_dim, dev)
    kind = _dtype_code(k.dtype, "k")
    if v.dtype != k.dtype or v.shape[0] != k.shape[0]:
        raise ValueError("k and v must have one dtype and one token count")
    batch = _batch4(starts, lens, table, dev)
    if rope is None:
        if positions is not None:
            raise ValueError("positions are the rope's: give one")
        _launch("dq_cache4_append", dev, load().dq_cache4_append, cache._struct(), batch, k.data_ptr(),
                v.data_ptr(), kind, k.shape[0], ks, vs)
        return
    if positions is not None:
        positions = _positions(positions, k.shape[0], dev)
    _launch("dq_cache4_append_rope", dev, load().dq_cache4_append_rope, cache._struct(), batch,
            k.data_ptr(), v.data_ptr(), kind, k.shape[0], ks, vs, rope._struct(dev), positions)


def cache4_read(cache: Cache4, tokens: int, starts, lens, table, dtype=None, k=None, v=None):
    """The dequantized (k, v) [tokens, kv_heads, D] of a call's tokens, float32 (the default)
    or bfloat16; rows of no sequence are left as they were."""
    torch = _torch()
    dev = cache.device_index
    kind = torch.float32 if dtype is None else dtype
    code = _dtype_code(kind, "dtype")
    shape = (tokens, cache.kv_heads, cache.head_dim)
    out = []
    for t, name in ((k, "k"), (v, "v")):
        if t is None:
            t = cache.k_codes.new_empty(shape, dtype=kind)
        else:
            _fast_need(t, name, kind, 3, dev)
            if tuple(t.shape) != shape:
                raise ValueError("%s must be [tokens, kv_heads, D]" % name)
        out.append(t)
    batch = _batch4(starts, lens, table, dev)
    _launch("dq_cache4_read", dev, load().dq_cache4_read, cache._struct(), batch, out[0].data_ptr(),
            out[1].data_ptr(), code, tokens)
    return tuple(out)


def cache4_attention(cache: Cache4, q, starts, lens, table, scale=None, max_q=None, max_len=None,
                     out=None, workspace=None):
    """Causal attention of q [tokens, q_heads, D] (bfloat16; tokens may be strided) over the
    cache, its tokens' keys and values already appended.  scale: D ** -0.5 unless given.
    max_q / max_len: the most new / cached tokens of a sequence, for sizing the launch
    (default: an even share of the call's tokens / the whole table); max_q = 1 (max_q * q_heads /
    kv_heads < 64) keeps the codes exact for prompts too, only slower.  out bfloat16 [tokens,
    q_heads, D]; workspace: uint8 tensor to use instead of a new one."""
    torch = _torch()
    dev = cache.device_index
    _gpu_index(q, "q")
    if q.dtype is not torch.bfloat16 or q.dim() != 3:
        raise TypeError("q must be a bfloat16 [tokens, q_heads, D] tensor")
    tokens, heads, D = q.shape
    stride = _token_rows(q, "q", heads, cache.head_dim, dev)
    batch = _batch4(starts, lens, table, dev)
    if out is None:
        out = q.new_empty((tokens, heads, D))
    else:
        _fast_need(out, "out", torch.bfloat16, 3, dev)
        if tuple(out.shape) != (tokens, heads, D):
            raise ValueError("out must be [tokens, q_heads, D]")
    if max_q is None:
        max_q = -(-tokens // max(batch.count, 1))
    if max_len is None:
        max_len = batch.table_width * cache.page_size
    if scale is None:
        scale = D ** -0.5
    lib = load()
    c = cache._struct()
    need = lib.dq_cache4_attention_workspace(c, batch.count, tokens, heads, max_q, max_len)
    if workspace is None:
        if need:
            workspace = q.new_empty((need,), dtype=torch.uint8)
    else:
        _fast_need(workspace, "workspace", torch.uint8, 1, dev)
        need = workspace.shape[0]
    _launch("dq_cache4_attention", dev, lib.dq_cache4_attention, c, batch, q.data_ptr(), tokens,
            stride, heads, scale, max_q, max_len, out.data_ptr(),
            workspace.data_ptr() if workspace is not None else None, need)
    return out


def draft_tree(parents, starts, lens=None, words=None):
    """What a tree of drafted tokens needs: (mask int32 [tokens, words], positions int32 [tokens]).
    parents int32 [tokens]: each token's parent, counted within its sequence's rows (starts int32
    [count + 1]), an earlier row, -1 for a root (as a sequence's rows from 4096 on are).  Bit j % 32 of mask word j / 32 says that the token
    sees its sequence's row j: itself or an ancestor.  words: the most rows of a sequence / 32,
    rounded up (default: enough for any sequence, tokens / 32).  positions: with ``lens`` (cached tokens, the rows
    included), where to rotate each: the context's length plus the row's depth; else None.  Rows of no
    sequence are left as allocated: zeros."""
    torch = _torch()
    dev = _gpu_index(parents, "parents")
    _fast_need(parents, "parents", torch.int32, 1, dev)
    _fast_need(starts, "starts", torch.int32, 1, dev)
    tokens, count = parents.shape[0], starts.shape[0] - 1
    if words is None:
        words = -(-tokens // 32)
    if not 1 <= words <= 65536:
        raise DQError(DQ_ERR_SHAPE, "draft_tree")
    mask = parents.new_zeros((tokens, words))
    positions = None
    if lens is not None:
        _fast_need(lens, "lens", torch.int32, 1, dev)
        if lens.shape[0] != count:
            raise ValueError("starts must be [count + 1], lens [count]")
        positions = parents.new_zeros((tokens,))
    _launch("dq_draft_tree", dev, load().dq_draft_tree, parents.data_ptr(), starts.data_ptr(),
            lens.data_ptr() if lens is not None else None, count, tokens, words, mask.data_ptr(),
            positions.data_ptr() if positions is not None else None)
    return mask, positions


def cache4_tree_attention(cache: Cache4, q, starts, lens, table, mask, scale=None, max_q=None,
                          max_len=None, out=None, workspace=None):
    """``cache4_attention`` for trees of drafted tokens: a token sees the cached positions before
    the call's own and, of its sequence's rows, those with a bit in mask int32 [tokens, words]
    (``draft_tree`` makes it; any bits will do).  The other arguments as there."""
    torch = _torch()
    dev = cache.device_index
    _gpu_index(q, "q")
    if q.dtype is not torch.bfloat16 or q.dim() != 3:
        raise TypeError("q must be a bfloat16 [tokens, q_heads, D] tensor")
    tokens, heads, D = q.shape
    stride = _token_rows(q, "q", heads, cache.head_dim, dev)
    batch = _batch4(starts, lens, table, dev)
    _fast_need(mask, "mask", torch.int32, 2, dev)
    if mask.shape[0] != tokens:
        raise ValueError("mask must be [tokens, words]")
    if out is None:
        out = q.new_empty((tokens, heads, D))
    else:
        _fast_need(out, "out", torch.bfloat16, 3, dev)
        if tuple(out.shape) != (tokens, heads, D):
            raise ValueError("out must be [tokens, q_heads, D]")
    if max_q is None:
        max_q = -(-tokens // max(batch.count, 1))
    if max_len is None:
        max_len = batch.table_width * cache.page_size
    if scale is None:
        scale = D ** -0.5
    lib = load()
    c = cache._struct()
    need = lib.dq_cache4_tree_attention_workspace(c, batch.count, tokens, heads, max_q, max_len)
    if workspace is None:
        if need:
            workspace = q.new_empty((need,), dtype=torch.uint8)
    else:
        _fast_need(workspace, "workspace", torch.uint8, 1, dev)
        need = workspace.shape[0]
    _launch("dq_cache4_tree_attention", dev, lib.dq_cache4_tree_attention, c, batch, q.data_ptr(), tokens,
            stride, heads, mask.data_ptr(), mask.shape[1], scale, max_q, max_len, out.data_ptr(),
            workspace.data_ptr() if workspace is not None else None, need)
    return out


def _prob_rows(t, name, tokens, vocab, dev):
    """Checks t float32 [tokens, vocab] (rows may be strided) on GPU ``dev``; returns its row stride."""
    torch = _torch()
    if _gpu_index(t, name) != dev:
        raise ValueError("%s: all tensors must be on one GPU (cuda:%d and %s)" % (name, dev, t.device))
    if t.dtype is not torch.float32:
        raise TypeError("%s must be float32 (got %s)" % (name, t.dtype))
    if t.dim() != 2 or t.shape[0] != tokens or (vocab is not None and t.shape[1] != vocab):
        raise ValueError("%s must be [tokens, vocab]" % name)
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s: a row must be contiguous" % name)
    return t.stride(0) if tokens > 1 else t.shape[1]


def verify_drafts(probs, ids, parents, starts, uniforms, draft_probs=None, workspace=None):
    """Verify drafted tokens against the target's probabilities: (path int32 [tokens], accepted int32
    [count], next int32 [count]).

    probs float32 [tokens, vocab]: the target's distribution of the token behind each row; ids,
    parents int32 [tokens]: the rows' tokens, and their parents as for ``draft_tree`` (row 0 of a sequence
    is its root, the last token known); starts int32 [count + 1]; uniforms float32 [tokens] in [0, 1).
    Without draft_probs a row's children are candidates of any origin, tried in order; with them
    (float32 [tokens, vocab]) a row's first child, drawn from its draft_probs, is tried alone.  The tokens
    that come out are distributed as the target's (the rule: ``dq_verify_drafts`` in include/dq.h).
    path: from starts[b] on, the accepted[b] rows of sequence b, its root first, then -1 (rows of no sequence:
    any value); next: the token drawn behind the last of them.  workspace: uint8 tensor to use instead of a new one."""
    torch = _torch()
    dev = _gpu_index(probs, "probs")
    _fast_need(ids, "ids", torch.int32, 1, dev)
    _fast_need(parents, "parents", torch.int32, 1, dev)
    _fast_need(starts, "starts", torch.int32, 1, dev)
    _fast_need(uniforms, "uniforms", torch.float32, 1, dev)
    tokens, count = ids.shape[0], starts.shape[0] - 1
    if parents.shape[0] != tokens or uniforms.shape[0] != tokens:
        raise ValueError("ids, parents and uniforms must be [tokens]")
    stride = _prob_rows(probs, "probs", tokens, None, dev)
    vocab = probs.shape[1]
    draft_stride = 0
    if draft_probs is not None:
        draft_stride = _prob_rows(draft_probs, "draft_probs", tokens, vocab, dev)
        draft_probs = draft_probs.data_ptr()
    lib = load()
    need = lib.dq_verify_drafts_workspace(count, vocab)
    if workspace is None:
        workspace = ids.new_empty((need,), dtype=torch.uint8)
    else:
        _fast_need(workspace, "workspace", torch.uint8, 1, dev)
        need = workspace.shape[0]
    path, accepted, drawn = ids.new_empty((tokens,)), ids.new_empty((count,)), ids.new_empty((count,))
    _launch("dq_verify_drafts", dev, lib.dq_verify_drafts, probs.data_ptr(), stride, draft_probs,
            draft_stride, ids.data_ptr(), parents.data_ptr(), starts.data_ptr(), uniforms.data_ptr(), tokens,
            count, vocab, path.data_ptr(), accepted.data_ptr(), drawn.data_ptr(), workspace.data_ptr(), need)
    return path, accepted, drawn


def cache4_keep(cache: Cache4, starts, lens, table, path, accepted) -> None:
    """Move the accepted rows' keys and values to the front of the call's own positions: of each
    sequence the rows path[starts[b]], path[starts[b] + 1], ... (``verify_drafts``' path int32 [tokens] and
    accepted int32 [count]).  It then has lens - rows + accepted tokens."""
    torch = _torch()
    dev = cache.device_index
    batch = _batch4(starts, lens, table, dev)
    _fast_need(path, "path", torch.int32, 1, dev)
    _fast_need(accepted, "accepted", torch.int32, 1, dev)
    if accepted.shape[0] != batch.count:
        raise ValueError("accepted must be [count]")
    _launch("dq_cache4_keep", dev, load().dq_cache4_keep, cache._struct(), batch, path.data_ptr(),
            accepted.data_ptr(), path.shape[0])


def stream_read(buf, nparts: int, partial=None):
    """Plain streaming read of a contiguous GPU tensor (any dtype, a multiple of
    16 bytes): the yardstick for the bandwidth-bound calls, not a step of the
    method.  Returns int32 [nparts] whose XOR is the XOR of every 32-bit word."""
    torch = _torch()
    if not isinstance(buf, torch.Tensor) or buf.device.type != "cuda" or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous GPU tensor")
    if partial is None:
        partial = torch.empty((nparts,), dtype=torch.int32, device=buf.device)
    _need(partial, "partial", (torch.int32,), 1)
    if partial.shape[0] != nparts:
        raise ValueError("partial must hold nparts words")
    nbytes = buf.numel() * buf.element_size()
    _check(dq_stream_read(buf.data_ptr(), nbytes, partial.data_ptr(), nparts, _stream(buf)),
           "dq_stream_read")
    return partial


# ------------------------------------------------------ on-disk packed format

def write_packed_file(path: str, matrices) -> None:
    """Write matrices to a packed-weight file.  ``matrices``: (name, N, K, bits,
    data, scales) with host numpy arrays -- data the packed words [N, row_words]
    (any 4-byte dtype) for bits 2..15, or bf16 bit patterns [N, K] (uint16) for
    bits 16; scales float32 [N] (None for bits 16)."""
    import numpy as np
    keep = []
    arr = (DQFileMatrix * len(matrices))()
    for i, (name, N, K, bits, data, scales) in enumerate(matrices):
        raw = name.encode("utf-8")
        if len(raw) > 63 or b"\0" in raw:
            raise ValueError("a name takes at most 63 UTF-8 bytes and no NUL")
        data = np.ascontiguousarray(data)
        want = N * (K * 2 if bits == 16 else dq_packed_row_bytes(K, bits))
        if data.nbytes != want:
            raise ValueError("matrix %r: data holds %d bytes, %d expected" % (name, data.nbytes, want))
        arr[i].name = raw
        arr[i].N, arr[i].K, arr[i].bits = N, K, bits
        arr[i].data = data.ctypes.data
        if scales is not None:
            scales = np.ascontiguousarray(scales, dtype=np.float32)
            if scales.shape != (N,):
                raise ValueError("matrix %r: scales must be float32 [N]" % name)
            arr[i].scales = scales.ctypes.data
        keep.append((data, scales))
    _check(int(load().dq_file_write(path.encode(), arr, len(matrices))), "dq_file_write")


class PackedFile:
    """A packed-weight file mapped read-only (``dq_file_open``); use as a
    context manager or call ``close``."""

    def __init__(self, path: str):
        h = ctypes.c_void_p()
        _check(int(load().dq_file_open(path.encode(), ctypes.byref(h))), "dq_file_open")
        self._h = h

    def __len__(self):
        return int(load().dq_file_count(self._h))

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def close(self):
        if self._h:
            load().dq_file_close(self._h)
            self._h = ctypes.c_void_p()

    def info(self, i: int):
        """(name, N, K, bits, data, scales): numpy views into the mapping (valid
        until ``close``); data is uint32 [N, row_words] or uint16 (bf16) [N, K]."""
        import numpy as np
        m = DQFileMatrix()
        _check(int(load().dq_file_matrix_info(self._h, i, ctypes.byref(m))), "dq_file_matrix_info")
        N, K, bits = int(m.N), int(m.K), int(m.bits)
        if bits == 16:
            data = np.ctypeslib.as_array(ctypes.cast(m.data, ctypes.POINTER(ctypes.c_uint16)),
                                         shape=(N, K))
            scales = None
        else:
            rw = dq_packed_row_bytes(K, bits) // 4
            data = np.ctypeslib.as_array(ctypes.cast(m.data, ctypes.POINTER(ctypes.c_uint32)),
                                         shape=(N, rw))
            scales = np.ctypeslib.as_array(ctypes.cast(m.scales, ctypes.POINTER(ctypes.c_float)),
                                           shape=(N,))
        return m.name.decode("utf-8"), N, K, bits, data, scales

    def verify(self, i: int) -> bool:
        st = int(load().dq_file_verify(self._h, i))
        if st == DQ_ERR_FORMAT:
            return False
        _check(st, "dq_file_verify")
        return True

    def load(self, i: int, device="cuda"):
        """Copy entry i into new GPU tensors: (packed int32 [N, row_words], scales
        float32 [N]) for bits 2..15, (bf16 [N, K], None) for bits 16.  Waits for
        the copy, so the tensors are ready when it returns."""
        torch = _torch()
        name, N, K, bits, _, _ = self.info(i)
        dev = torch.device(device)
        if bits == 16:
            data = torch.empty((N, K), dtype=torch.bfloat16, device=dev)
            scales = None
        else:
            data = torch.empty((N, dq_packed_row_bytes(K, bits) // 4), dtype=torch.int32, device=dev)
            scales = torch.empty((N,), dtype=torch.float32, device=dev)
        stream = torch.cuda.current_stream(dev)
        _check(int(load().dq_file_load(self._h, i, data.data_ptr(),
                                       scales.data_ptr() if scales is not None else 0,
                                       stream.cuda_stream)), "dq_file_load")
        stream.synchronize()
        return data, scales
