"""Whole steps of the hot path, composed from the C entry points.

A step is the pages' sequence -- score the blocks, keep the top-k (with the
current / last block), attend over the kept blocks -- issued as consecutive
library calls on one stream.  Buffers are allocated once (torch is only the
device-memory provider here) and reused, so a step launches kernels and
nothing else.
"""
from __future__ import annotations

import contextlib
import math
from dataclasses import dataclass, field
from typing import ClassVar, Dict, Optional, Tuple

import torch

from . import (bsa_gated_attn_bwd, bsa_workspace_bytes_bwd, BSA_OP_DECODE, BSA_OP_DECODE_HEADS, BSA_OP_GIST_DECODE, BSA_SCORE_DECODE,
               BSA_SCORE_DECODE_HEADS, BSA_SCORE_PREFILL, BSA_TOPK_CAUSAL_BLOCK, bsa_decode_select,
               bsa_gated_attn_fwd, bsa_gist_expand_decode, bsa_score_blocks, bsa_sparse_attn_decode,
               bsa_hssa_decode, bsa_paged_append, bsa_sparse_attn_decode_heads, bsa_workspace_bytes_hssa, bsa_sparse_attn_decode_paged, bsa_sparse_attn_prefill,
               bsa_topk_select, bsa_topk_select_joint_heads, bsa_topk_select_pattern, bsa_workspace_bytes,
               make_shape, BSA_OP_DECODE_QUANT, BSA_ROPE_HALF, BSA_ROPE_NONE, bsa_paged_append_quant,
               bsa_paged_read_quant, bsa_qkv_norm_rope, bsa_qkv_norm_rope_bwd, bsa_sparse_attn_decode_quant,
               bsa_topk_select_lens, bsa_workspace_bytes_norm_rope, make_rope)


def _dev(t: torch.Tensor):
    return t.device


@dataclass
class PrefillStep:
    """pool+score -> top-k -> sparse (or gated) attention for q [B,Hq,N,d], k/v [B,Hkv,N,d].

    pattern=(sink, local) keeps, besides the kb best blocks, the first `sink`
    blocks and the `local` most recent ones (MInference block-sparse); the
    default keeps the current block only."""
    q: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor
    block: int
    kb: int
    gated: bool = False
    softmax_scale: Optional[float] = None
    pattern: Optional[Tuple[int, int]] = None
    bufs: Dict[str, torch.Tensor] = field(default_factory=dict)

    def __post_init__(self):
        B, Hq, N, d = self.q.shape
        Hkv = self.k.shape[1]
        nb = N // self.block
        self.shape = make_shape(B, Hq, Hkv, N, N, d, self.block, self.q.dtype)
        self.nb = nb
        self.idx_stride = self.kb + 1 if self.pattern is None else self.kb + self.pattern[0] + self.pattern[1]
        if self.softmax_scale is None:
            self.softmax_scale = 1.0 / math.sqrt(d)
        dev = _dev(self.q)
        f32 = torch.float32
        b = self.bufs
        b.setdefault("qbar", torch.empty((B, Hkv, nb, d), dtype=f32, device=dev))
        b.setdefault("kbar", torch.empty((B, Hkv, nb, d), dtype=f32, device=dev))
        b.setdefault("scores", torch.empty((B, Hkv, nb, nb), dtype=f32, device=dev))
        b.setdefault("idx", torch.empty((B, Hkv, nb, self.idx_stride), dtype=torch.int32, device=dev))
        b.setdefault("count", torch.empty((B, Hkv, nb), dtype=torch.int32, device=dev))
        b.setdefault("o", torch.empty_like(self.q))
        b.setdefault("lse", torch.empty((B, Hq, N), dtype=f32, device=dev))

    def select(self, stream=None):
        b = self.bufs
        bsa_score_blocks(self.shape, BSA_SCORE_PREFILL, self.q, self.k, None, b["qbar"], b["kbar"],
                         b["scores"], stream=stream)
        rows = self.shape.B * self.shape.Hkv * self.nb
        if self.pattern is None:
            bsa_topk_select(b["scores"], rows, self.nb, BSA_TOPK_CAUSAL_BLOCK, self.kb, b["idx"], self.idx_stride,
                            b["count"], stream=stream)
        else:
            sink, local = self.pattern
            bsa_topk_select_pattern(b["scores"], rows, self.nb, sink, local, self.kb, b["idx"], self.idx_stride,
                                    b["count"], stream=stream)

    def attend(self, idx: Optional[torch.Tensor] = None, stream=None, with_lse: bool = True):
        b = self.bufs
        idx = b["idx"] if idx is None else idx
        lse = b["lse"] if with_lse else None
        if self.gated:
            bsa_gated_attn_fwd(self.shape, self.q, self.k, self.v, idx, idx.shape[-1], b["scores"],
                               self.softmax_scale, b["o"], lse, stream=stream)
        else:
            bsa_sparse_attn_prefill(self.shape, self.q, self.k, self.v, idx, idx.shape[-1], self.softmax_scale,
                                    b["o"], lse, stream=stream)

    def run(self, stream=None, with_lse: bool = True):
        self.select(stream)
        self.attend(stream=stream, with_lse=with_lse)
        return self.bufs

    def backward(self, d_o: torch.Tensor, idx: Optional[torch.Tensor] = None, stream=None):
        """Gradients of sum(d_o * O) for the last attend() (run with its LSE):
        fp32 dq, dk, dv and, gated, dsel (the selector scores' gradient)."""
        b = self.bufs
        idx = b["idx"] if idx is None else idx
        dev = _dev(self.q)
        f32 = torch.float32
        b.setdefault("dq", torch.empty(self.q.shape, dtype=f32, device=dev))
        b.setdefault("dk", torch.empty(self.k.shape, dtype=f32, device=dev))
        b.setdefault("dv", torch.empty(self.v.shape, dtype=f32, device=dev))
        if self.gated:
            b.setdefault("dsel", torch.empty(b["scores"].shape, dtype=f32, device=dev))
        ws = bsa_workspace_bytes_bwd(self.shape, idx.shape[-1])
        if "bwd_workspace" not in b or b["bwd_workspace"].numel() < ws:
            b["bwd_workspace"] = torch.empty((max(ws, 256),), dtype=torch.uint8, device=dev)
        bsa_gated_attn_bwd(self.shape, self.q, self.k, self.v, b["lse"], d_o, idx, idx.shape[-1],
                           b["scores"] if self.gated else None, self.softmax_scale, b["dq"], b["dk"], b["dv"],
                           b["dsel"] if self.gated else None, b["bwd_workspace"], stream=stream)
        return b


@dataclass
class DecodeStep:
    """score (against the resident pooled-key summary) -> top-k -> split-K sparse decode.

    q [B,Hq,d]; k_cache/v_cache [B,Hkv,Nk,d]; kbar [B,Hkv,nb,d] fp32 is the
    block-mean summary kept next to the cache (built once by ``pool_cache``).
    """
    q: torch.Tensor
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    block: int
    kb: int
    softmax_scale: Optional[float] = None
    bufs: Dict[str, torch.Tensor] = field(default_factory=dict)

    def __post_init__(self):
        B, Hq, d = self.q.shape
        Hkv, Nk = self.k_cache.shape[1], self.k_cache.shape[2]
        nb = Nk // self.block
        self.nb = nb
        self.shape = make_shape(B, Hq, Hkv, 1, Nk, d, self.block, self.q.dtype)
        self.idx_stride = self.kb + 1
        if self.softmax_scale is None:
            self.softmax_scale = 1.0 / math.sqrt(d)
        dev = _dev(self.q)
        f32 = torch.float32
        b = self.bufs
        b.setdefault("kbar", torch.empty((B, Hkv, nb, d), dtype=f32, device=dev))
        b.setdefault("qbar", torch.empty((B, Hkv, d), dtype=f32, device=dev))
        b.setdefault("scores", torch.empty((B, Hkv, nb), dtype=f32, device=dev))
        b.setdefault("idx", torch.empty((B, Hkv, self.idx_stride), dtype=torch.int32, device=dev))
        b.setdefault("count", torch.empty((B, Hkv), dtype=torch.int32, device=dev))
        ws = bsa_workspace_bytes(BSA_OP_DECODE, self.shape, self.idx_stride)
        b.setdefault("workspace", torch.empty((max(ws, 256),), dtype=torch.uint8, device=dev))
        b.setdefault("o", torch.empty_like(self.q))
        b.setdefault("lse", torch.empty((B, Hq), dtype=f32, device=dev))

    def pool_cache(self, stream=None):
        """Build the pooled-key summary from the cache (off the per-step path)."""
        b = self.bufs
        bsa_score_blocks(self.shape, BSA_SCORE_DECODE, self.q, self.k_cache, None, b["qbar"], b["kbar"],
                         b["scores"], stream=stream)

    def select(self, stream=None):
        b = self.bufs
        bsa_decode_select(self.shape, self.q, b["kbar"], self.kb, b["scores"], b["idx"], self.idx_stride,
                          pooled_q_out=b["qbar"], count_out=b["count"], stream=stream)

    def attend(self, idx: Optional[torch.Tensor] = None, stream=None, with_lse: bool = True):
        b = self.bufs
        idx = b["idx"] if idx is None else idx
        bsa_sparse_attn_decode(self.shape, self.q, self.k_cache, self.v_cache, idx, idx.shape[-1],
                               self.softmax_scale, b["workspace"], b["o"], b["lse"] if with_lse else None,
                               stream=stream)

    def run(self, stream=None, with_lse: bool = True):
        self.select(stream)
        self.attend(stream=stream, with_lse=with_lse)
        return self.bufs


@dataclass
class GistStep:
    """SSA decode: gist scores -> per-head top-k chunks -> mixed attention (one C call)."""
    q: torch.Tensor
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    gist_k: torch.Tensor
    gist_v: torch.Tensor
    chunk: int
    topk: int
    softmax_scale: Optional[float] = None
    bufs: Dict[str, torch.Tensor] = field(default_factory=dict)

    def __post_init__(self):
        B, Hq, d = self.q.shape
        Hkv, Nk = self.k_cache.shape[1], self.k_cache.shape[2]
        self.shape = make_shape(B, Hq, Hkv, 1, Nk, d, self.chunk, self.q.dtype)
        if self.softmax_scale is None:
            self.softmax_scale = 1.0 / math.sqrt(d)
        dev = _dev(self.q)
        b = self.bufs
        ws = bsa_workspace_bytes(BSA_OP_GIST_DECODE, self.shape, self.topk)
        b.setdefault("workspace", torch.empty((max(ws, 256),), dtype=torch.uint8, device=dev))
        b.setdefault("idx", torch.empty((B, Hq, max(self.topk, 1)), dtype=torch.int32, device=dev))
        b.setdefault("o", torch.empty_like(self.q))
        b.setdefault("lse", torch.empty((B, Hq), dtype=torch.float32, device=dev))

    def run(self, idx_in: Optional[torch.Tensor] = None, stream=None, with_lse: bool = True):
        b = self.bufs
        bsa_gist_expand_decode(self.shape, self.q, self.k_cache, self.v_cache, self.gist_k, self.gist_v,
                               self.topk, idx_in, b["idx"] if self.topk > 0 else None, self.softmax_scale,
                               b["workspace"], b["o"], b["lse"] if with_lse else None, stream=stream)
        return b


@dataclass
class HeadBudgetDecodeStep:
    """Decode with one budget shared by the query heads of each KV group
    (Ada-KV): per-head scores against the pooled-key summary -> the best
    kb_total (head, block) pairs of the group, the last block kept by every
    head -> attention with each head's own kept blocks."""
    q: torch.Tensor
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    block: int
    kb_total: int
    softmax_scale: Optional[float] = None
    bufs: Dict[str, torch.Tensor] = field(default_factory=dict)

    def __post_init__(self):
        B, Hq, d = self.q.shape
        Hkv, Nk = self.k_cache.shape[1], self.k_cache.shape[2]
        nb = Nk // self.block
        self.nb = nb
        self.G = Hq // Hkv
        self.shape = make_shape(B, Hq, Hkv, 1, Nk, d, self.block, self.q.dtype)
        self.idx_stride = min(self.kb_total, nb - 1) + 1
        if self.softmax_scale is None:
            self.softmax_scale = 1.0 / math.sqrt(d)
        dev = _dev(self.q)
        f32 = torch.float32
        b = self.bufs
        b.setdefault("kbar", torch.empty((B, Hkv, nb, d), dtype=f32, device=dev))
        b.setdefault("qbar", torch.empty((B, Hkv, d), dtype=f32, device=dev))
        b.setdefault("scores", torch.empty((B, Hq, nb), dtype=f32, device=dev))
        b.setdefault("idx", torch.empty((B, Hq, self.idx_stride), dtype=torch.int32, device=dev))
        b.setdefault("count", torch.empty((B, Hq), dtype=torch.int32, device=dev))
        ws = bsa_workspace_bytes(BSA_OP_DECODE_HEADS, self.shape, self.idx_stride)
        b.setdefault("workspace", torch.empty((max(ws, 256),), dtype=torch.uint8, device=dev))
        b.setdefault("o", torch.empty_like(self.q))
        b.setdefault("lse", torch.empty((B, Hq), dtype=f32, device=dev))

    def pool_cache(self, stream=None):
        b = self.bufs
        group_scores = torch.empty((self.shape.B, self.shape.Hkv, self.nb), dtype=torch.float32, device=self.q.device)
        bsa_score_blocks(self.shape, BSA_SCORE_DECODE, self.q, self.k_cache, None, b["qbar"], b["kbar"],
                         group_scores, stream=stream)

    def select(self, stream=None):
        b = self.bufs
        bsa_score_blocks(self.shape, BSA_SCORE_DECODE_HEADS, self.q, None, b["kbar"], None, None, b["scores"],
                         stream=stream)
        bsa_topk_select_joint_heads(b["scores"], self.shape.B * self.shape.Hkv, self.G, self.nb, self.kb_total,
                                    b["idx"], self.idx_stride, b["count"], stream=stream)

    def attend(self, idx: Optional[torch.Tensor] = None, stream=None, with_lse: bool = True):
        b = self.bufs
        idx = b["idx"] if idx is None else idx
        bsa_sparse_attn_decode_heads(self.shape, self.q, self.k_cache, self.v_cache, idx, idx.shape[-1],
                                     self.softmax_scale, b["workspace"], b["o"], b["lse"] if with_lse else None,
                                     stream=stream)

    def run(self, stream=None, with_lse: bool = True):
        self.select(stream)
        self.attend(stream=stream, with_lse=with_lse)
        return self.bufs


@dataclass
class PagedDecodeStep:
    """Decode over a paged KV cache (PagedAttention): pools [P,Hkv,64,d] of
    physical blocks and a block table [B, nb] mapping each sequence's logical
    blocks to them.  The pooled-key summary [B,Hkv,nb,d] is kept by
    ``append`` (each block is pooled when it completes); ``select`` scores
    the query against it and keeps the top-kb logical blocks with the last;
    ``attend`` gathers the kept blocks through the table."""
    q: torch.Tensor
    k_pool: torch.Tensor
    v_pool: torch.Tensor
    block_table: torch.Tensor
    block: int
    kb: int
    softmax_scale: Optional[float] = None
    bufs: Dict[str, torch.Tensor] = field(default_factory=dict)

    def __post_init__(self):
        B, Hq, d = self.q.shape
        Hkv = self.k_pool.shape[1]
        nb = self.block_table.shape[1]
        self.nb = nb
        self.shape = make_shape(B, Hq, Hkv, 1, nb * self.block, d, self.block, self.q.dtype)
        self.idx_stride = self.kb + 1
        if self.softmax_scale is None:
            self.softmax_scale = 1.0 / math.sqrt(d)
        dev = _dev(self.q)
        f32 = torch.float32
        b = self.bufs
        b.setdefault("kbar", torch.zeros((B, Hkv, nb, d), dtype=f32, device=dev))
        b.setdefault("qbar", torch.empty((B, Hkv, d), dtype=f32, device=dev))
        b.setdefault("scores", torch.empty((B, Hkv, nb), dtype=f32, device=dev))
        b.setdefault("idx", torch.empty((B, Hkv, self.idx_stride), dtype=torch.int32, device=dev))
        b.setdefault("count", torch.empty((B, Hkv), dtype=torch.int32, device=dev))
        ws = bsa_workspace_bytes(BSA_OP_DECODE, self.shape, self.idx_stride)
        b.setdefault("workspace", torch.empty((max(ws, 256),), dtype=torch.uint8, device=dev))
        b.setdefault("o", torch.empty_like(self.q))
        b.setdefault("lse", torch.empty((B, Hq), dtype=f32, device=dev))

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, seq_lens: torch.Tensor, stream=None):
        """Write k_new/v_new [B,Hkv,T,d] after seq_lens[b] tokens; completed blocks are pooled."""
        B, Hkv, T, d = k_new.shape
        shape = make_shape(B, Hkv, Hkv, T, self.nb * self.block, d, self.block, k_new.dtype)
        bsa_paged_append(shape, k_new, v_new, seq_lens, self.block_table, self.k_pool, self.v_pool,
                         self.bufs["kbar"], stream=stream)

    def select(self, stream=None):
        b = self.bufs
        bsa_decode_select(self.shape, self.q, b["kbar"], self.kb, b["scores"], b["idx"], self.idx_stride,
                          pooled_q_out=b["qbar"], count_out=b["count"], stream=stream)

    def attend(self, idx: Optional[torch.Tensor] = None, stream=None, with_lse: bool = True):
        b = self.bufs
        idx = b["idx"] if idx is None else idx
        bsa_sparse_attn_decode_paged(self.shape, self.q, self.k_pool, self.v_pool, self.block_table, idx,
                                     idx.shape[-1], self.softmax_scale, b["workspace"], b["o"],
                                     b["lse"] if with_lse else None, stream=stream)

    def run(self, stream=None, with_lse: bool = True):
        self.select(stream)
        self.attend(stream=stream, with_lse=with_lse)
        return self.bufs


@dataclass
class HssaStep:
    """Two-level gist routing decode (H-SSA): meta-gist scores -> km groups
    per head -> gist scores inside them -> topk chunks per head -> attention
    over expanded tokens, gists of kept groups, meta-gists of the rest (one C
    call).  Groups are 64 chunks; meta_k/meta_v [B,Hkv,nc/64,d]."""
    q: torch.Tensor
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    gist_k: torch.Tensor
    gist_v: torch.Tensor
    meta_k: torch.Tensor
    meta_v: torch.Tensor
    chunk: int
    km: int
    topk: int
    softmax_scale: Optional[float] = None
    bufs: Dict[str, torch.Tensor] = field(default_factory=dict)

    def __post_init__(self):
        B, Hq, d = self.q.shape
        Hkv, Nk = self.k_cache.shape[1], self.k_cache.shape[2]
        self.shape = make_shape(B, Hq, Hkv, 1, Nk, d, self.chunk, self.q.dtype)
        if self.softmax_scale is None:
            self.softmax_scale = 1.0 / math.sqrt(d)
        dev = _dev(self.q)
        b = self.bufs
        ws = bsa_workspace_bytes_hssa(self.shape, self.km, self.topk)
        b.setdefault("workspace", torch.empty((max(ws, 256),), dtype=torch.uint8, device=dev))
        b.setdefault("meta_idx", torch.empty((B, Hq, self.km), dtype=torch.int32, device=dev))
        b.setdefault("idx", torch.empty((B, Hq, max(self.topk, 1)), dtype=torch.int32, device=dev))
        b.setdefault("o", torch.empty_like(self.q))
        b.setdefault("lse", torch.empty((B, Hq), dtype=torch.float32, device=dev))

    def run(self, stream=None, with_lse: bool = True):
        b = self.bufs
        bsa_hssa_decode(self.shape, self.q, self.k_cache, self.v_cache, self.gist_k, self.gist_v, self.meta_k,
                        self.meta_v, self.km, self.topk, b["meta_idx"], b["idx"] if self.topk > 0 else None,
                        self.softmax_scale, b["workspace"], b["o"], b["lse"] if with_lse else None, stream=stream)
        return b


def _fits(what: str, t: Optional[torch.Tensor], shape: Tuple[int, ...]):
    if t is not None and t.shape != shape:
        raise ValueError(f"{what} is {list(shape)}, got {list(t.shape)}")


def _buffer(bufs: Dict[str, torch.Tensor], name: str, shape, dtype, device, zero: bool = False):
    """Makes the buffer of that name, or checks that the caller's own is large enough."""
    if name not in bufs:
        bufs[name] = (torch.zeros if zero else torch.empty)(shape, dtype=dtype, device=device)
    elif bufs[name].numel() < math.prod(shape):
        raise ValueError(f"bufs[{name!r}] is {list(shape)}, got {list(bufs[name].shape)}")


def _memory_of(stream):
    """Memory taken inside belongs to the call's stream: taken on the current one it may still be in use there, by work
    that the call's stream does not wait for."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


class _Replaceable:
    """A step whose fields may be replaced between calls: at the next one those replaced are checked, against the sizes
    that the step was built for (``_sizes``), and what is derived from them is derived again (``_derive``)."""
    _stale: ClassVar[Tuple[str, ...]] = ()

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name not in self._stale:
            object.__setattr__(self, "_stale", self._stale + (name,))

    def _bring_up(self, stream=None):
        others = []
        for name in self._stale:
            size = self._sizes.get(name)
            if size is None:
                others.append(name)
            else:
                _fits(name, getattr(self, name), size)
        if others:
            self._derive(others, stream)
        object.__setattr__(self, "_stale", ())


@dataclass
class QkvStep(_Replaceable):
    """From a fused projection qkv [B,N,Hq+2Hkv,d] to q [B,Hq,N,d], k and v [B,Hkv,N,d] for the steps here: RMS
    norm of every query and key head (q_weight and k_weight [d], or None), rotation by position, head-major order.

    inv_freq: float64 [rot_dim/2] on the device (bsa_rope_inv_freq; None: no rotation); positions [B,N] int32 or
    None (0..N-1); rope_scale: the factor of a scaling for long contexts.  A field replaced by another of its size
    counts from the next call on.  For decode (N = 1), q is bufs["q"][:, :, 0] and k, v are PagedDecodeStep.append's or
    QuantDecodeStep.append's k_new, v_new."""
    qkv: torch.Tensor
    Hq: int
    Hkv: int
    q_weight: Optional[torch.Tensor] = None
    k_weight: Optional[torch.Tensor] = None
    eps: float = 1e-6
    inv_freq: Optional[torch.Tensor] = None
    layout: int = BSA_ROPE_HALF
    positions: Optional[torch.Tensor] = None
    rope_scale: float = 1.0
    bufs: Dict[str, torch.Tensor] = field(default_factory=dict)

    def __post_init__(self):
        B, N, H, d = self.qkv.shape
        if H != self.Hq + 2 * self.Hkv:
            raise ValueError(f"qkv has {H} heads a token, not {self.Hq} + 2 * {self.Hkv}")
        self.shape = make_shape(B, self.Hq, self.Hkv, N, N, d, 1, self.qkv.dtype)
        self._sizes = {"qkv": (B, N, H, d), "positions": (B, N), "q_weight": (d,), "k_weight": (d,)}
        self._bring_up()

    def _derive(self, stale, stream):
        s = self.shape
        if (self.Hq, self.Hkv) != (s.Hq, s.Hkv):
            raise ValueError(f"this step has {s.Hq} query and {s.Hkv} key heads")
        if "inv_freq" in stale or "layout" in stale or "rope_scale" in stale:
            self.rope = make_rope(self.layout if self.inv_freq is not None else BSA_ROPE_NONE, self.inv_freq,
                                  self.rope_scale)
        if "bufs" in stale:
            with _memory_of(stream):
                for name, heads in (("q", s.Hq), ("k", s.Hkv), ("v", s.Hkv)):
                    _buffer(self.bufs, name, (s.B, heads, s.Nq, s.d), self.qkv.dtype, self.qkv.device)

    def run(self, stream=None):
        if self._stale:
            self._bring_up(stream)
        b = self.bufs
        bsa_qkv_norm_rope(self.shape, self.qkv, self.q_weight, self.k_weight, self.eps, self.rope, self.positions,
                          b["q"], b["k"], b["v"], stream=stream)
        return b

    def backward(self, dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor, stream=None):
        """Gradients d_qkv (qkv's type, dense) and, with weights, d_q_weight and d_k_weight (fp32) from fp32 dq, dk,
        dv, as PrefillStep.backward gives them."""
        if self._stale:
            self._bring_up(stream)
        B, N, H, d = self.qkv.shape
        for name, g, heads in (("dq", dq, self.Hq), ("dk", dk, self.Hkv), ("dv", dv, self.Hkv)):
            if g.shape != (B, heads, N, d):
                raise ValueError(f"{name} is [{B}, {heads}, {N}, {d}], got {list(g.shape)}")
        b = self.bufs
        dev = self.qkv.device
        if "d_qkv" not in b:
            with _memory_of(stream):
                b["d_qkv"] = torch.empty((B, N, H, d), dtype=self.qkv.dtype, device=dev)
        weights = (None, None, None)
        if self.q_weight is not None:
            if "d_q_weight" not in b or "d_k_weight" not in b or "qkv_workspace" not in b:
                with _memory_of(stream):
                    _buffer(b, "d_q_weight", (d,), torch.float32, dev)
                    _buffer(b, "d_k_weight", (d,), torch.float32, dev)
                    if "qkv_workspace" not in b:
                        b["qkv_workspace"] = torch.empty((bsa_workspace_bytes_norm_rope(self.shape),),
                                                         dtype=torch.uint8, device=dev)
            weights = (b["d_q_weight"], b["d_k_weight"], b["qkv_workspace"])
            if weights[0].numel() < d or weights[1].numel() < d:
                raise ValueError(f"bufs['d_q_weight'] and bufs['d_k_weight'] are [{d}]")
        bsa_qkv_norm_rope_bwd(self.shape, self.qkv, self.q_weight, self.k_weight, self.eps, self.rope, self.positions,
                              dq, dk, dv, b["d_qkv"], *weights, stream=stream)
        return b


@dataclass
class QuantDecodeStep(_Replaceable):
    """Decode over a paged KV cache of 8 bits whose sequences have their own lengths: pools [P,Hkv,64,d] of e4m3
    codes, exponents [P,Hkv,64], a block table [B, nb] and seq_lens [B] (int32, the tokens each sequence holds;
    the caller advances them after ``append``).  ``append`` quantises new tokens and pools completed blocks;
    ``select`` scores the query against the pooled summary and keeps each sequence's kb best history blocks and
    its last; ``attend`` gathers them through the table.  kb None: every block is attended, nothing is selected.
    ``read`` gives tokens back as dense rows.  A field may be replaced by another of its size."""
    q: torch.Tensor
    k_pool: torch.Tensor
    v_pool: torch.Tensor
    k_exp: torch.Tensor
    v_exp: torch.Tensor
    block_table: torch.Tensor
    seq_lens: torch.Tensor
    kb: Optional[int] = None
    softmax_scale: Optional[float] = None
    bufs: Dict[str, torch.Tensor] = field(default_factory=dict)

    def __post_init__(self):
        B, Hq, d = self.q.shape
        Hkv, block = self.k_pool.shape[1], self.k_pool.shape[2]
        nb = self.block_table.shape[1]
        if self.k_pool.shape[3] != d or self.block_table.shape[0] != B or self.seq_lens.shape != (B,) or \
                Hq % Hkv != 0:
            raise ValueError("q [B,Hq,d], pools [P,Hkv,64,d], block_table [B,nb] and seq_lens [B] do not match")
        self.nb, self.block = nb, block
        self.shape = make_shape(B, Hq, Hkv, 1, nb * block, d, block, self.q.dtype)
        self.idx_stride = 0 if self.kb is None else self.kb + 1
        if self.softmax_scale is None:
            self.softmax_scale = 1.0 / math.sqrt(d)
        self._sizes = {"q": (B, Hq, d), "block_table": (B, nb), "seq_lens": (B,)}
        self._bring_up()

    def _derive(self, stale, stream):
        s = self.shape
        if "k_pool" in stale:      # the other pools are compared with it at every call
            _fits("k_pool", self.k_pool, (self.k_pool.shape[0], s.Hkv, self.block, s.d))
        if (self.kb is None) != (self.idx_stride == 0) or (self.kb is not None and self.kb >= self.idx_stride):
            raise ValueError(f"this step was built for kb {f'< {self.idx_stride}' if self.idx_stride else 'None'}, "
                             f"got {self.kb}")
        if "bufs" in stale:
            with _memory_of(stream):
                self._buffers()

    def _buffers(self):
        s, b, dev, f32 = self.shape, self.bufs, _dev(self.q), torch.float32
        if self.idx_stride:
            _buffer(b, "kbar", (s.B, s.Hkv, self.nb, s.d), f32, dev, zero=True)
            _buffer(b, "qbar", (s.B, s.Hkv, s.d), f32, dev)
            _buffer(b, "scores", (s.B, s.Hkv, self.nb), f32, dev)
            _buffer(b, "idx", (s.B, s.Hkv, self.idx_stride), torch.int32, dev)
            _buffer(b, "count", (s.B, s.Hkv), torch.int32, dev)
        if "workspace" not in b:
            ws = bsa_workspace_bytes(BSA_OP_DECODE_QUANT, s, self.idx_stride)
            b["workspace"] = torch.empty((max(ws, 256),), dtype=torch.uint8, device=dev)
        _buffer(b, "o", (s.B, s.Hq, s.d), self.q.dtype, dev)
        _buffer(b, "lse", (s.B, s.Hq), f32, dev)

    def _rows_shape(self, T: int, dtype):
        s = self.shape
        return make_shape(s.B, s.Hkv, s.Hkv, T, s.Nk, s.d, s.block, dtype)

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, new_lens: Optional[torch.Tensor] = None, stream=None):
        """Quantise k_new/v_new [B,Hkv,T,d] (t < new_lens[b]) behind seq_lens[b] tokens; completed blocks are pooled."""
        if self._stale:
            self._bring_up(stream)
        s = self.shape
        if k_new.shape != v_new.shape or k_new.shape[:2] != (s.B, s.Hkv) or k_new.shape[3] != s.d:
            raise ValueError(f"new keys and values are [{s.B}, {s.Hkv}, T, {s.d}], got {list(k_new.shape)}")
        if new_lens is not None and new_lens.shape != (s.B,):
            raise ValueError(f"new_lens is [{s.B}], got {list(new_lens.shape)}")
        bsa_paged_append_quant(self._rows_shape(k_new.shape[2], k_new.dtype), k_new, v_new, self.seq_lens,
                               self.block_table, self.k_pool, self.v_pool, self.k_exp, self.v_exp,
                               self.bufs.get("kbar"), new_lens=new_lens, stream=stream)

    def read(self, k_out: torch.Tensor, v_out: torch.Tensor, starts: Optional[torch.Tensor] = None, stream=None):
        """Tokens starts[b] + t into row t of k_out/v_out [B,Hkv,T,d] (bf16 or fp32), as far as the sequence goes."""
        if self._stale:
            self._bring_up(stream)
        s = self.shape
        if k_out.shape != v_out.shape or k_out.shape[:2] != (s.B, s.Hkv) or k_out.shape[3] != s.d:
            raise ValueError(f"rows read back are [{s.B}, {s.Hkv}, T, {s.d}], got {list(k_out.shape)}")
        if starts is not None and starts.shape != (s.B,):
            raise ValueError(f"starts is [{s.B}], got {list(starts.shape)}")
        bsa_paged_read_quant(self._rows_shape(k_out.shape[2], k_out.dtype), self.k_pool, self.v_pool, self.k_exp,
                             self.v_exp, self.block_table, self.seq_lens, k_out, v_out, starts=starts, stream=stream)

    def select(self, stream=None):
        if self._stale:
            self._bring_up(stream)
        if self.kb is None:
            raise ValueError("this step attends every block (kb None): there is nothing to select")
        b, s = self.bufs, self.shape
        bsa_score_blocks(s, BSA_SCORE_DECODE, self.q, None, b["kbar"], b["qbar"], None, b["scores"], stream=stream)
        bsa_topk_select_lens(b["scores"], s.B * s.Hkv, self.nb, self.seq_lens, s.Hkv, self.block, self.kb, b["idx"],
                             self.idx_stride, b["count"], stream=stream)

    def attend(self, idx: Optional[torch.Tensor] = None, stream=None, with_lse: bool = True):
        if self._stale:
            self._bring_up(stream)
        b = self.bufs
        if idx is None:
            idx = b["idx"] if self.kb is not None else None
        elif idx.dim() != 3 or idx.shape[0] != self.shape.B or idx.shape[1] != self.shape.Hkv:
            raise ValueError(f"idx is [{self.shape.B}, {self.shape.Hkv}, n], got {list(idx.shape)}")
        bsa_sparse_attn_decode_quant(self.shape, self.q, self.k_pool, self.v_pool, self.k_exp, self.v_exp,
                                     self.block_table, self.seq_lens, idx, 0 if idx is None else idx.shape[-1],
                                     self.softmax_scale, b["workspace"], b["o"], b["lse"] if with_lse else None,
                                     stream=stream)
        return b

    def run(self, stream=None, with_lse: bool = True):
        if self.kb is not None:
            self.select(stream)
        return self.attend(stream=stream, with_lse=with_lse)
