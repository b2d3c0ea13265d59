"""Python binding of libbsa, the B200 (sm_100a) library for query-aware
top-k block-sparse causal attention.

Argument marshalling only: every function here forwards torch tensors'
device pointers and the current CUDA stream to the C entry point of the same
name declared in ``include/bsa.h``; all computation runs in the library's
CUDA kernels.  There is no CPU fallback: importing the package fails if
``libbsa.so`` has not been built (``python top_block_sparse_bsa_b200/_build.py``).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

__all__ = [
    "BsaError", "BsaShape", "lib", "LIB_PATH",
    "BSA_F32", "BSA_BF16",
    "BSA_SCORE_PREFILL", "BSA_SCORE_DECODE", "BSA_SCORE_GIST", "BSA_SCORE_DECODE_HEADS",
    "BSA_TOPK_CAUSAL_BLOCK", "BSA_TOPK_LAST_BLOCK", "BSA_TOPK_PLAIN",
    "BSA_OP_DECODE", "BSA_OP_GIST_DECODE", "BSA_OP_DECODE_HEADS",
    "make_shape", "bsa_score_blocks", "bsa_topk_select", "bsa_sparse_attn_prefill",
    "bsa_gated_attn_fwd", "bsa_sparse_attn_decode", "bsa_gist_expand_decode",
    "bsa_workspace_bytes", "bsa_status_string", "bsa_device_status", "bsa_version",
    "bsa_sparse_attn_decode_noalloc", "bsa_decode_split_override", "bsa_selftest_wait_expiry",
    "bsa_prefill_kernel_override", "bsa_decode_select", "bsa_topk_select_pattern",
    "bsa_topk_select_joint_heads", "bsa_sparse_attn_decode_heads", "bsa_sparse_attn_decode_paged",
    "bsa_paged_append", "bsa_hssa_decode", "bsa_workspace_bytes_hssa", "bsa_gated_attn_bwd",
    "bsa_workspace_bytes_bwd", "EXPORTED_SYMBOLS",
    "BSA_OP_DECODE_QUANT", "BSA_ROPE_NONE", "BSA_ROPE_HALF", "BSA_ROPE_PAIRS", "BSA_ROPE_PLAIN", "BSA_ROPE_LINEAR",
    "BSA_ROPE_BASE", "BSA_ROPE_PARTS", "BsaRope", "make_rope", "bsa_rope_inv_freq", "bsa_qkv_norm_rope",
    "bsa_qkv_norm_rope_bwd", "bsa_workspace_bytes_norm_rope", "bsa_paged_append_quant", "bsa_paged_read_quant",
    "bsa_sparse_attn_decode_quant", "bsa_topk_select_lens",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libbsa.so")

BSA_OK, BSA_ERR_INVALID_ARG, BSA_ERR_UNSUPPORTED, BSA_ERR_CUDA, BSA_ERR_TIMEOUT, BSA_ERR_DEVICE = range(6)
BSA_F32, BSA_BF16 = 0, 1
BSA_SCORE_PREFILL, BSA_SCORE_DECODE, BSA_SCORE_GIST, BSA_SCORE_DECODE_HEADS = 0, 1, 2, 3
BSA_TOPK_CAUSAL_BLOCK, BSA_TOPK_LAST_BLOCK, BSA_TOPK_PLAIN = 0, 1, 2
BSA_OP_DECODE, BSA_OP_GIST_DECODE, BSA_OP_DECODE_HEADS, BSA_OP_DECODE_QUANT = 0, 1, 2, 3
BSA_ROPE_NONE, BSA_ROPE_HALF, BSA_ROPE_PAIRS = 0, 1, 2
BSA_ROPE_PLAIN, BSA_ROPE_LINEAR, BSA_ROPE_BASE, BSA_ROPE_PARTS = 0, 1, 2, 3

# Every symbol the C header declares.
EXPORTED_SYMBOLS = (
    "bsa_score_blocks", "bsa_topk_select", "bsa_sparse_attn_prefill", "bsa_gated_attn_fwd",
    "bsa_sparse_attn_decode", "bsa_gist_expand_decode", "bsa_workspace_bytes",
    "bsa_status_string", "bsa_device_status", "bsa_version", "bsa_sparse_attn_decode_noalloc",
    "bsa_decode_split_override", "bsa_selftest_wait_expiry", "bsa_prefill_kernel_override",
    "bsa_decode_select", "bsa_topk_select_pattern", "bsa_topk_select_joint_heads", "bsa_sparse_attn_decode_heads",
    "bsa_sparse_attn_decode_paged", "bsa_paged_append", "bsa_hssa_decode", "bsa_workspace_bytes_hssa",
    "bsa_gated_attn_bwd", "bsa_workspace_bytes_bwd", "bsa_rope_inv_freq", "bsa_qkv_norm_rope",
    "bsa_qkv_norm_rope_bwd", "bsa_workspace_bytes_norm_rope", "bsa_paged_append_quant", "bsa_paged_read_quant",
    "bsa_sparse_attn_decode_quant", "bsa_topk_select_lens",
)


class BsaError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} failed: {_status_name(code)}")


class BsaShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("Nq", ctypes.c_int),
                ("Nk", ctypes.c_int), ("d", ctypes.c_int), ("block", ctypes.c_int), ("dtype", ctypes.c_int)]

    def __repr__(self):
        return (f"BsaShape(B={self.B}, Hq={self.Hq}, Hkv={self.Hkv}, Nq={self.Nq}, Nk={self.Nk}, "
                f"d={self.d}, block={self.block}, dtype={self.dtype})")


class BsaRope(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int), ("rot_dim", ctypes.c_int), ("inv_freq", ctypes.c_void_p),
                ("scale", ctypes.c_float)]
    freq = None      # the tensor behind inv_freq, where make_rope made this


_p = ctypes.c_void_p
_i = ctypes.c_int
_d = ctypes.c_double
_ll = ctypes.c_longlong
_f = ctypes.c_float
_SIGS = {
    "bsa_score_blocks": (_i, [ctypes.POINTER(BsaShape), _i, _p, _p, _p, _p, _p, _p, _p]),
    "bsa_topk_select": (_i, [_p, _i, _i, _i, _i, _p, _i, _p, _p]),
    "bsa_decode_select": (_i, [ctypes.POINTER(BsaShape), _p, _p, _i, _p, _p, _p, _i, _p, _p]),
    "bsa_topk_select_pattern": (_i, [_p, _i, _i, _i, _i, _i, _p, _i, _p, _p]),
    "bsa_sparse_attn_decode_paged": (_i, [ctypes.POINTER(BsaShape), _p, _p, _p, _i, _p, _i, _p, _i, ctypes.c_float,
                                          _p, ctypes.c_size_t, _p, _p, _p]),
    "bsa_paged_append": (_i, [ctypes.POINTER(BsaShape), _p, _p, _p, _p, _i, _i, _p, _p, _p, _p]),
    "bsa_hssa_decode": (_i, [ctypes.POINTER(BsaShape), _p, _p, _p, _p, _p, _p, _p, _i, _i, _p, _p, ctypes.c_float,
                             _p, ctypes.c_size_t, _p, _p, _p]),
    "bsa_workspace_bytes_hssa": (ctypes.c_size_t, [ctypes.POINTER(BsaShape), _i, _i]),
    "bsa_gated_attn_bwd": (_i, [ctypes.POINTER(BsaShape), _p, _p, _p, _p, _p, _p, _i, _p, ctypes.c_float, _p, _p,
                                _p, _p, _p, ctypes.c_size_t, _p]),
    "bsa_workspace_bytes_bwd": (ctypes.c_size_t, [ctypes.POINTER(BsaShape), _i]),
    "bsa_topk_select_joint_heads": (_i, [_p, _i, _i, _i, _i, _p, _i, _p, _p]),
    "bsa_sparse_attn_decode_heads": (_i, [ctypes.POINTER(BsaShape), _p, _p, _p, _p, _i, ctypes.c_float, _p,
                                          ctypes.c_size_t, _p, _p, _p]),
    "bsa_sparse_attn_prefill": (_i, [ctypes.POINTER(BsaShape), _p, _p, _p, _p, _i, ctypes.c_float, _p, _p, _p]),
    "bsa_gated_attn_fwd": (_i, [ctypes.POINTER(BsaShape), _p, _p, _p, _p, _i, _p, ctypes.c_float, _p, _p, _p]),
    "bsa_sparse_attn_decode": (_i, [ctypes.POINTER(BsaShape), _p, _p, _p, _p, _i, ctypes.c_float, _p,
                                    ctypes.c_size_t, _p, _p, _p]),
    "bsa_gist_expand_decode": (_i, [ctypes.POINTER(BsaShape), _p, _p, _p, _p, _p, _i, _p, _p, ctypes.c_float,
                                    _p, ctypes.c_size_t, _p, _p, _p]),
    "bsa_sparse_attn_decode_noalloc": (_i, [ctypes.POINTER(BsaShape), _p, _p, _p, _p, _i, ctypes.c_float, _p,
                                            _p, _p]),
    "bsa_workspace_bytes": (ctypes.c_size_t, [_i, ctypes.POINTER(BsaShape), _i]),
    "bsa_status_string": (ctypes.c_char_p, [_i]),
    "bsa_device_status": (_i, [ctypes.POINTER(ctypes.c_uint), _i]),
    "bsa_version": (_i, []),
    "bsa_decode_split_override": (_i, [_i]),
    "bsa_prefill_kernel_override": (_i, [_i]),
    "bsa_selftest_wait_expiry": (_i, [ctypes.c_longlong, _p]),
    "bsa_rope_inv_freq": (_i, [_i, _d, _i, _d, _d, _d, _d, _p, _p]),
    "bsa_qkv_norm_rope": (_i, [ctypes.POINTER(BsaShape), _p, _ll, _p, _p, _f, ctypes.POINTER(BsaRope), _p, _p, _p, _p,
                               _p]),
    "bsa_qkv_norm_rope_bwd": (_i, [ctypes.POINTER(BsaShape), _p, _ll, _p, _p, _f, ctypes.POINTER(BsaRope), _p, _p, _p,
                                   _p, _p, _ll, _p, _p, _p, ctypes.c_size_t, _p]),
    "bsa_workspace_bytes_norm_rope": (ctypes.c_size_t, [ctypes.POINTER(BsaShape)]),
    "bsa_paged_append_quant": (_i, [ctypes.POINTER(BsaShape), _p, _p, _p, _p, _p, _i, _i, _p, _p, _p, _p, _p, _p]),
    "bsa_paged_read_quant": (_i, [ctypes.POINTER(BsaShape), _p, _p, _p, _p, _i, _p, _i, _p, _p, _p, _p, _p]),
    "bsa_sparse_attn_decode_quant": (_i, [ctypes.POINTER(BsaShape), _p, _p, _p, _p, _p, _i, _p, _i, _p, _p, _i, _f, _p,
                                          ctypes.c_size_t, _p, _p, _p]),
    "bsa_topk_select_lens": (_i, [_p, _i, _i, _p, _i, _i, _i, _p, _i, _p, _p]),
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libbsa.so is not built at {LIB_PATH}; build it with "
                          "`python top_block_sparse_bsa_b200/_build.py`")
    L = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGS.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


lib = _load()


def _status_name(code: int) -> str:
    return lib.bsa_status_string(code).decode()


def _check(fn: str, code: int) -> None:
    if code != BSA_OK:
        raise BsaError(fn, code)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libbsa takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libbsa takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BSA_BF16
    if t.dtype == torch.float32:
        return BSA_F32
    raise ValueError(f"unsupported dtype {t.dtype}")


def make_shape(B, Hq, Hkv, Nq, Nk, d, block, dtype) -> BsaShape:
    if isinstance(dtype, torch.dtype):
        dtype = BSA_BF16 if dtype == torch.bfloat16 else BSA_F32
    try:
        return BsaShape(B, Hq, Hkv, Nq, Nk, d, block, dtype)
    except TypeError:      # numbers that are no Python ints
        return BsaShape(int(B), int(Hq), int(Hkv), int(Nq), int(Nk), int(d), int(block), int(dtype))


def bsa_version() -> int:
    return int(lib.bsa_version())


def bsa_status_string(code: int) -> str:
    return _status_name(code)


def bsa_device_status(reset: bool = False):
    """(status code, flag bits) of the current device; synchronises it."""
    flags = ctypes.c_uint(0)
    code = lib.bsa_device_status(ctypes.byref(flags), 1 if reset else 0)
    return int(code), int(flags.value)


def bsa_decode_split_override(num_splits: int) -> int:
    """Fix the decode split-K range count (> 0) or restore the default (<= 0); returns the previous setting."""
    return int(lib.bsa_decode_split_override(int(num_splits)))


def bsa_prefill_kernel_override(kernel: int) -> int:
    """Force a bf16 prefill kernel (1 paired tiles, 2 one tile per SM, 3 SM pair) or 0 for the
    shape's default; returns the previous setting."""
    return int(lib.bsa_prefill_kernel_override(int(kernel)))


def bsa_selftest_wait_expiry(budget_cycles: int, stream=None) -> None:
    """Enqueue the bounded-wait expiry self-test kernel (sets BSA_DEV_TIMEOUT in the status word)."""
    _check("bsa_selftest_wait_expiry", lib.bsa_selftest_wait_expiry(int(budget_cycles), _stream(stream)))


def bsa_workspace_bytes(op: int, shape: BsaShape, budget: int) -> int:
    return int(lib.bsa_workspace_bytes(op, ctypes.byref(shape), int(budget)))


def bsa_score_blocks(shape: BsaShape, mode: int, q, k=None, pooled_k_in=None, pooled_q_out=None,
                     pooled_k_out=None, scores=None, stream=None) -> None:
    _check("bsa_score_blocks", lib.bsa_score_blocks(
        ctypes.byref(shape), int(mode), _ptr(q), _ptr(k), _ptr(pooled_k_in), _ptr(pooled_q_out),
        _ptr(pooled_k_out), _ptr(scores), _stream(stream)))


def bsa_topk_select(scores, rows: int, ncols: int, mode: int, kb: int, idx_out, idx_stride: int,
                    count_out=None, stream=None) -> None:
    _check("bsa_topk_select", lib.bsa_topk_select(
        _ptr(scores), int(rows), int(ncols), int(mode), int(kb), _ptr(idx_out), int(idx_stride),
        _ptr(count_out), _stream(stream)))


def bsa_topk_select_pattern(scores, rows: int, ncols: int, sink: int, local: int, kb: int, idx_out,
                            idx_stride: int, count_out=None, stream=None) -> None:
    _check("bsa_topk_select_pattern", lib.bsa_topk_select_pattern(
        _ptr(scores), int(rows), int(ncols), int(sink), int(local), int(kb), _ptr(idx_out), int(idx_stride),
        _ptr(count_out), _stream(stream)))


def bsa_topk_select_joint_heads(scores, rows: int, heads: int, ncols: int, kb_total: int, idx_out,
                                idx_stride: int, count_out=None, stream=None) -> None:
    _check("bsa_topk_select_joint_heads", lib.bsa_topk_select_joint_heads(
        _ptr(scores), int(rows), int(heads), int(ncols), int(kb_total), _ptr(idx_out), int(idx_stride),
        _ptr(count_out), _stream(stream)))


def bsa_sparse_attn_decode_heads(shape: BsaShape, q, k_cache, v_cache, idx, idx_stride: int, softmax_scale: float,
                                 workspace, o, lse=None, stream=None) -> None:
    _check("bsa_sparse_attn_decode_heads", lib.bsa_sparse_attn_decode_heads(
        ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(idx), int(idx_stride),
        ctypes.c_float(softmax_scale), _ptr(workspace), ctypes.c_size_t(workspace.numel() * workspace.element_size()),
        _ptr(o), _ptr(lse), _stream(stream)))


def bsa_sparse_attn_decode_paged(shape: BsaShape, q, k_pool, v_pool, block_table, idx, idx_stride: int,
                                 softmax_scale: float, workspace, o, lse=None, stream=None) -> None:
    """Decode over a paged cache: pools [P,Hkv,64,d], block_table [B, table_stride]."""
    _check("bsa_sparse_attn_decode_paged", lib.bsa_sparse_attn_decode_paged(
        ctypes.byref(shape), _ptr(q), _ptr(k_pool), _ptr(v_pool), int(k_pool.shape[0]), _ptr(block_table),
        int(block_table.shape[-1]), _ptr(idx), int(idx_stride), ctypes.c_float(softmax_scale), _ptr(workspace),
        ctypes.c_size_t(workspace.numel() * workspace.element_size()), _ptr(o), _ptr(lse), _stream(stream)))


def bsa_paged_append(shape: BsaShape, k_new, v_new, seq_lens, block_table, k_pool, v_pool, pooled_k=None,
                     stream=None) -> None:
    """Write k_new/v_new [B,Hkv,T,d] at positions seq_lens[b]+t of the paged cache; pool completed blocks."""
    _check("bsa_paged_append", lib.bsa_paged_append(
        ctypes.byref(shape), _ptr(k_new), _ptr(v_new), _ptr(seq_lens), _ptr(block_table), int(block_table.shape[-1]),
        int(k_pool.shape[0]), _ptr(k_pool), _ptr(v_pool), _ptr(pooled_k), _stream(stream)))


def bsa_hssa_decode(shape: BsaShape, q, k_cache, v_cache, gist_k, gist_v, meta_k, meta_v, km: int, topk: int,
                    meta_out=None, idx_out=None, softmax_scale: float = 0.0, workspace=None, o=None, lse=None,
                    stream=None) -> None:
    _check("bsa_hssa_decode", lib.bsa_hssa_decode(
        ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(gist_k), _ptr(gist_v), _ptr(meta_k),
        _ptr(meta_v), int(km), int(topk), _ptr(meta_out), _ptr(idx_out), ctypes.c_float(softmax_scale),
        _ptr(workspace), ctypes.c_size_t(workspace.numel() * workspace.element_size() if workspace is not None else 0),
        _ptr(o), _ptr(lse), _stream(stream)))


def bsa_workspace_bytes_hssa(shape: BsaShape, km: int, topk: int) -> int:
    return int(lib.bsa_workspace_bytes_hssa(ctypes.byref(shape), int(km), int(topk)))


def bsa_gated_attn_bwd(shape: BsaShape, q, k, v, lse, d_o, idx, idx_stride: int, sel_scores, softmax_scale: float,
                       dq, dk, dv, dsel=None, workspace=None, stream=None) -> None:
    """Backward of the sparse (sel_scores None) or gated prefill attention: fp32 dq, dk, dv (and dsel)."""
    _check("bsa_gated_attn_bwd", lib.bsa_gated_attn_bwd(
        ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(lse), _ptr(d_o), _ptr(idx), int(idx_stride),
        _ptr(sel_scores), ctypes.c_float(softmax_scale), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dsel), _ptr(workspace),
        ctypes.c_size_t(workspace.numel() * workspace.element_size() if workspace is not None else 0),
        _stream(stream)))


def bsa_workspace_bytes_bwd(shape: BsaShape, idx_stride: int) -> int:
    return int(lib.bsa_workspace_bytes_bwd(ctypes.byref(shape), int(idx_stride)))


def bsa_decode_select(shape: BsaShape, q, pooled_k, kb: int, scores, idx_out, idx_stride: int,
                      pooled_q_out=None, count_out=None, stream=None) -> None:
    _check("bsa_decode_select", lib.bsa_decode_select(
        ctypes.byref(shape), _ptr(q), _ptr(pooled_k), int(kb), _ptr(pooled_q_out), _ptr(scores), _ptr(idx_out),
        int(idx_stride), _ptr(count_out), _stream(stream)))


def bsa_sparse_attn_prefill(shape: BsaShape, q, k, v, idx, idx_stride: int, softmax_scale: float, o,
                            lse=None, stream=None) -> None:
    _check("bsa_sparse_attn_prefill", lib.bsa_sparse_attn_prefill(
        ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(idx), int(idx_stride),
        ctypes.c_float(softmax_scale), _ptr(o), _ptr(lse), _stream(stream)))


def bsa_gated_attn_fwd(shape: BsaShape, q, k, v, idx, idx_stride: int, sel_scores, softmax_scale: float, o,
                       lse=None, stream=None) -> None:
    _check("bsa_gated_attn_fwd", lib.bsa_gated_attn_fwd(
        ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(idx), int(idx_stride), _ptr(sel_scores),
        ctypes.c_float(softmax_scale), _ptr(o), _ptr(lse), _stream(stream)))


def bsa_sparse_attn_decode(shape: BsaShape, q, k_cache, v_cache, idx, idx_stride: int, softmax_scale: float,
                           workspace, o, lse=None, stream=None) -> None:
    _check("bsa_sparse_attn_decode", lib.bsa_sparse_attn_decode(
        ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(idx), int(idx_stride),
        ctypes.c_float(softmax_scale), _ptr(workspace), ctypes.c_size_t(workspace.numel() * workspace.element_size()),
        _ptr(o), _ptr(lse), _stream(stream)))


def bsa_gist_expand_decode(shape: BsaShape, q, k_cache, v_cache, gist_k, gist_v, topk: int, idx_in=None,
                           idx_out=None, softmax_scale: float = 0.0, workspace=None, o=None, lse=None,
                           stream=None) -> None:
    _check("bsa_gist_expand_decode", lib.bsa_gist_expand_decode(
        ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(gist_k), _ptr(gist_v), int(topk),
        _ptr(idx_in), _ptr(idx_out), ctypes.c_float(softmax_scale), _ptr(workspace),
        ctypes.c_size_t(workspace.numel() * workspace.element_size() if workspace is not None else 0),
        _ptr(o), _ptr(lse), _stream(stream)))


def bsa_sparse_attn_decode_noalloc(shape: BsaShape, q, k_cache, v_cache, idx, idx_stride: int,
                                   softmax_scale: float, o, lse=None, stream=None) -> None:
    """Decode without a caller-provided workspace (scratch lives in the library)."""
    _check("bsa_sparse_attn_decode_noalloc", lib.bsa_sparse_attn_decode_noalloc(
        ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(idx), int(idx_stride),
        ctypes.c_float(softmax_scale), _ptr(o), _ptr(lse), _stream(stream)))


def make_rope(layout: int, inv_freq=None, scale: float = 1.0) -> Optional[BsaRope]:
    """Rotation of the first 2*len(inv_freq) channels (inv_freq: float64 on the device, held by the result); None for
    BSA_ROPE_NONE."""
    if layout == BSA_ROPE_NONE:
        if inv_freq is not None:
            raise ValueError("BSA_ROPE_NONE takes no frequencies")
        return None
    if inv_freq is None:
        raise ValueError("a rotation needs its frequencies")
    if inv_freq.dtype != torch.float64:
        raise ValueError(f"inv_freq is float64, got {inv_freq.dtype}")
    rope = BsaRope(int(layout), 2 * inv_freq.numel(), _ptr(inv_freq), float(scale))
    rope.freq = inv_freq
    return rope


def bsa_rope_inv_freq(rot_dim: int, base: float = 10000.0, scaling: int = BSA_ROPE_PLAIN, factor: float = 1.0,
                      original_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(frequencies [rot_dim/2] float64 on the host, factor on the rotated values)."""
    out = torch.empty((max(int(rot_dim), 0) // 2,), dtype=torch.float64)
    scale = ctypes.c_float(0.0)
    _check("bsa_rope_inv_freq", lib.bsa_rope_inv_freq(
        int(rot_dim), float(base), int(scaling), float(factor), float(original_len), float(beta_fast),
        float(beta_slow), ctypes.c_void_p(out.data_ptr() if out.numel() else None), ctypes.byref(scale)))
    return out, float(scale.value)


# What the calls below check of a tensor before its pointer goes to the library: its type, that it is dense, and that it
# lives on the device that the call runs on, the current one.  One pass over each tensor: a decode step is a few
# microseconds on the device, so the binding counts.

def _at(what: str, t, dtype, device: int):
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        _refuse(what, t, dtype, device)
    return t.data_ptr()


def _refuse(what: str, t, dtype, device: int):
    if not t.is_cuda:
        raise ValueError(f"{what}: libbsa takes device tensors")
    if t.dtype is not dtype:
        raise ValueError(f"{what} is {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{what} is on {t.device}, the call runs on cuda:{device}")
    raise ValueError(f"{what}: libbsa takes contiguous tensors")


def _here(stream):
    """(current device, stream handle on it)."""
    device = torch._C._cuda_getDevice()
    if stream is None:
        return device, torch._C._cuda_getCurrentRawStream(device)
    return device, _stream(stream)


def _token_rows(what: str, x, shape: BsaShape, dtype, device: int):
    """Pointer and token stride of x [B, Nq, Hq+2Hkv, d]: dense but for the distance between tokens."""
    if x.dtype is not dtype or x.get_device() != device:
        _refuse(what, x, dtype, device)
    size, heads, d = x.size(), shape.Hq + 2 * shape.Hkv, shape.d
    if size != (shape.B, shape.Nq, heads, d):
        raise ValueError(f"{what} is [{shape.B}, {shape.Nq}, {heads}, {d}], got {list(size)}")
    if x.is_contiguous():
        return x.data_ptr(), heads * d
    stride = x.stride()
    token = stride[1] if shape.Nq > 1 else (stride[0] if shape.B > 1 else heads * d)
    if (d > 1 and stride[3] != 1) or (heads > 1 and stride[2] != d) or \
            (shape.B > 1 and stride[0] != shape.Nq * token):
        raise ValueError(f"{what}: heads and channels are dense, tokens evenly apart")
    return x.data_ptr(), token


def _rope_at(rope: Optional[BsaRope], device: int):
    """The library's argument for a rotation, its frequencies checked as every tensor is."""
    if rope is None:
        return None
    freq = rope.freq
    if freq is not None:
        if freq.get_device() != device or freq.data_ptr() != rope.inv_freq:
            rope.inv_freq = _at("inv_freq", freq, torch.float64, device)
    return ctypes.byref(rope)


def _size(t) -> int:
    return t.numel() * t.element_size() if t is not None else 0


def bsa_workspace_bytes_norm_rope(shape: BsaShape) -> int:
    return int(lib.bsa_workspace_bytes_norm_rope(ctypes.byref(shape)))


def bsa_qkv_norm_rope(shape: BsaShape, qkv, q_weight, k_weight, eps: float, rope: Optional[BsaRope], positions,
                      q, k, v, stream=None) -> None:
    """Norms, rotation and change to head-major of qkv [B, Nq, Hq+2Hkv, d] (a slice of wider rows may be given)."""
    dev, st = _here(stream)
    t = qkv.dtype
    src, token_stride = _token_rows("qkv", qkv, shape, t, dev)
    code = lib.bsa_qkv_norm_rope(
        ctypes.byref(shape), src, token_stride, _at("q_weight", q_weight, t, dev), _at("k_weight", k_weight, t, dev),
        eps, _rope_at(rope, dev), _at("positions", positions, torch.int32, dev),
        _at("q", q, t, dev), _at("k", k, t, dev), _at("v", v, t, dev), st)
    if code:
        raise BsaError("bsa_qkv_norm_rope", code)


def bsa_qkv_norm_rope_bwd(shape: BsaShape, qkv, q_weight, k_weight, eps: float, rope: Optional[BsaRope], positions,
                          dq, dk, dv, d_qkv, d_q_weight=None, d_k_weight=None, workspace=None, stream=None) -> None:
    """Gradients of qkv and of the norms' weights from fp32 dq, dk, dv."""
    dev, st = _here(stream)
    t, f32 = qkv.dtype, torch.float32
    src, token_stride = _token_rows("qkv", qkv, shape, t, dev)
    dst, d_token_stride = _token_rows("d_qkv", d_qkv, shape, t, dev)
    code = lib.bsa_qkv_norm_rope_bwd(
        ctypes.byref(shape), src, token_stride, _at("q_weight", q_weight, t, dev), _at("k_weight", k_weight, t, dev),
        eps, _rope_at(rope, dev), _at("positions", positions, torch.int32, dev),
        _at("dq", dq, f32, dev), _at("dk", dk, f32, dev), _at("dv", dv, f32, dev), dst, d_token_stride,
        _at("d_q_weight", d_q_weight, f32, dev), _at("d_k_weight", d_k_weight, f32, dev),
        _at("workspace", workspace, torch.uint8, dev), _size(workspace), st)
    if code:
        raise BsaError("bsa_qkv_norm_rope_bwd", code)


def _quant_pools(k_pool, v_pool, k_exp, v_exp, device: int):
    """Pointers of pools [P,Hkv,64,d] (e4m3 codes) and exponents [P,Hkv,64]."""
    codes = k_pool.dtype
    if codes is not torch.float8_e4m3fn and codes is not torch.uint8:
        raise ValueError(f"pools hold e4m3 codes (float8_e4m3fn or uint8), got {codes}")
    size = k_pool.size()
    if v_pool.size() != size or k_exp.size() != size[:3] or v_exp.size() != size[:3]:
        raise ValueError("pools [P,Hkv,64,d] and exponents [P,Hkv,64] do not match")
    return (_at("k_pool", k_pool, codes, device), _at("v_pool", v_pool, codes, device),
            _at("k_exp", k_exp, torch.uint8, device), _at("v_exp", v_exp, torch.uint8, device), size[0])


def bsa_paged_append_quant(shape: BsaShape, k_new, v_new, seq_lens, block_table, k_pool, v_pool, k_exp, v_exp,
                           pooled_k=None, new_lens=None, stream=None) -> None:
    """Quantise k_new/v_new [B,Hkv,T,d] into positions seq_lens[b]+t (t < new_lens[b]) of the paged cache; pool
    completed blocks."""
    dev, st = _here(stream)
    i32, bf16 = torch.int32, torch.bfloat16
    kp, vp, ke, ve, pages = _quant_pools(k_pool, v_pool, k_exp, v_exp, dev)
    code = lib.bsa_paged_append_quant(
        ctypes.byref(shape), _at("k_new", k_new, bf16, dev), _at("v_new", v_new, bf16, dev),
        _at("seq_lens", seq_lens, i32, dev), _at("new_lens", new_lens, i32, dev),
        _at("block_table", block_table, i32, dev), block_table.size(-1), pages, kp, vp, ke, ve,
        _at("pooled_k", pooled_k, torch.float32, dev), st)
    if code:
        raise BsaError("bsa_paged_append_quant", code)


def bsa_paged_read_quant(shape: BsaShape, k_pool, v_pool, k_exp, v_exp, block_table, seq_lens, k_out, v_out,
                         starts=None, stream=None) -> None:
    """Tokens starts[b]+t of the quantised cache as dense rows [B,Hkv,T,d]; rows past a sequence stay as they were."""
    dev, st = _here(stream)
    i32, t = torch.int32, torch.bfloat16 if shape.dtype == BSA_BF16 else torch.float32
    kp, vp, ke, ve, pages = _quant_pools(k_pool, v_pool, k_exp, v_exp, dev)
    code = lib.bsa_paged_read_quant(
        ctypes.byref(shape), kp, vp, ke, ve, pages, _at("block_table", block_table, i32, dev), block_table.size(-1),
        _at("seq_lens", seq_lens, i32, dev), _at("starts", starts, i32, dev), _at("k_out", k_out, t, dev),
        _at("v_out", v_out, t, dev), st)
    if code:
        raise BsaError("bsa_paged_read_quant", code)


def bsa_sparse_attn_decode_quant(shape: BsaShape, q, k_pool, v_pool, k_exp, v_exp, block_table, seq_lens, idx,
                                 idx_stride: int, softmax_scale: float, workspace, o, lse=None, stream=None) -> None:
    """Decode over the quantised paged cache: kept blocks idx [B,Hkv,idx_stride], or every block (None, 0)."""
    dev, st = _here(stream)
    i32, bf16 = torch.int32, torch.bfloat16
    kp, vp, ke, ve, pages = _quant_pools(k_pool, v_pool, k_exp, v_exp, dev)
    code = lib.bsa_sparse_attn_decode_quant(
        ctypes.byref(shape), _at("q", q, bf16, dev), kp, vp, ke, ve, pages, _at("block_table", block_table, i32, dev),
        block_table.size(-1), _at("seq_lens", seq_lens, i32, dev), _at("idx", idx, i32, dev), idx_stride,
        softmax_scale, _at("workspace", workspace, torch.uint8, dev), _size(workspace), _at("o", o, bf16, dev),
        _at("lse", lse, torch.float32, dev), st)
    if code:
        raise BsaError("bsa_sparse_attn_decode_quant", code)


def bsa_topk_select_lens(scores, rows: int, ncols: int, lens, rows_per_len: int, block: int, kb: int, idx_out,
                         idx_stride: int, count_out=None, stream=None) -> None:
    """Decode selection where row r's sequence r // rows_per_len holds lens[r // rows_per_len] tokens."""
    dev, st = _here(stream)
    i32 = torch.int32
    code = lib.bsa_topk_select_lens(
        _at("scores", scores, torch.float32, dev), rows, ncols, _at("lens", lens, i32, dev), rows_per_len, block, kb,
        _at("idx_out", idx_out, i32, dev), idx_stride, _at("count_out", count_out, i32, dev), st)
    if code:
        raise BsaError("bsa_topk_select_lens", code)
