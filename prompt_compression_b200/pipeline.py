"""End-to-end compositions of the C entry points (allocation by torch only).

speckv_compress   scores -> pool + top-C_max + window -> compacted K/V
specpc_select     SpecPC scores -> pool + top-K prompt tokens
cascade_compress  SpecPC on the draft, gather the target K/V at the kept
                  tokens, then SpecKV on the gathered cache (SpecKV-PC)
PagedCache        the tensors of a paged KV cache, and its operators
speckv_compress_pages  SpecKV with the kept rows written straight into a
                  paged cache

"Draft-based Approximate Inference for LLMs" (paper notes), section 关键设计.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import binding as B


class SpeckvBuffers:
    """Preallocated outputs and scratch for repeated speckv_compress calls (on
    `stream`, if they are not to run on the current one)."""

    def __init__(self, q, k, v, n_window: int, c_max: int, window_mass: bool = False,
                 with_pooled: bool = False, stream=None):
        Bsz, L, hq, R, d = q.shape
        _, _, hkv, n_in, _ = k.shape
        units = Bsz * L * hkv
        n_pre = n_in - n_window
        keep = min(c_max, n_pre) + n_window
        shape = B.speckv_shape(q, k, n_window)

        def empty(size, dtype):
            return B._output_on(stream, q, size, dtype)

        self.units, self.n_pre, self.keep = units, n_pre, keep
        self.scores = empty((units, n_pre), torch.float32)
        self.window_mass = empty((units, n_window), torch.float32) if window_mass else None
        self.pooled = empty((units, n_pre), torch.float32) if with_pooled else None
        self.idx = empty((units, keep), torch.int32)
        self.k_out = empty((Bsz, L, hkv, keep, d), k.dtype)
        self.v_out = empty((Bsz, L, hkv, keep, d), v.dtype) if v is not None else None
        self.ws_score = empty(max(B.speckv_workspace_size(shape), 256), torch.uint8)
        self.ws_topk = empty(max(B.topk_workspace_size(units, n_pre), 256), torch.uint8)


def speckv_compress(q, k, v, n_window: int, c_max: int, pool: int = 7, scale: float = 1.0,
                    buffers: Optional[SpeckvBuffers] = None, window_mass: bool = False, stream=None,
                    pool_mode: int = B.SPK_POOL_MAX):
    """SpecKV on every unit: returns the buffers object (scores, idx, k_out, v_out).
    pool_mode: B.SPK_POOL_MAX (the workloads' max pool) or B.SPK_POOL_AVG."""
    buf = buffers or SpeckvBuffers(q, k, v, n_window, c_max, window_mass=window_mass, stream=stream)
    B.speckv_score(q, k, n_window, buf.scores, buf.window_mass, buf.ws_score, scale, stream)
    B.topk_select(buf.scores, c_max, n_window, buf.idx, pool, buf.pooled, buf.ws_topk, stream, pool_mode)
    B.kv_compact(k, v, buf.idx, buf.k_out, buf.v_out, 1, stream)
    return buf


def specpc_select(q, k, row_weights, l_skip: int, keep: int, pool: int = 7, n_lookahead: int = 1,
                  scale: float = 1.0, scores=None, idx=None, stream=None, pool_mode: int = B.SPK_POOL_MAX):
    """SpecPC prompt-token selection: (scores [B, n_in], idx [B, min(keep, n_in)])."""
    Bsz = q.shape[0]
    n_in = k.shape[3]
    if scores is None:
        scores = B._output_on(stream, q, (Bsz, n_in), torch.float32)
    if idx is None:
        idx = B._output_on(stream, q, (Bsz, min(keep, n_in)), torch.int32)
    B.specpc_score(q, k, row_weights, scores, l_skip, n_lookahead, None, scale, stream)
    B.topk_select(scores, keep, 0, idx, pool, None, None, stream, pool_mode)
    return scores, idx


def cascade_compress(draft_q, draft_k, row_weights, l_skip: int, keep: int, target_q, target_k, target_v,
                     n_window: int, c_max: int, pool: int = 7, stream=None):
    """SpecKV-PC: SpecPC keeps `keep` prompt tokens, the target K/V are gathered
    at them (one index row per batch element, shared by every layer and KV
    head), then SpecKV keeps c_max + n_window of the gathered tokens."""
    Bsz, L, hkv, n_full, d = target_k.shape
    pc_scores, pc_idx = specpc_select(draft_q, draft_k, row_weights, l_skip, keep, pool, stream=stream)
    n_keep = pc_idx.shape[1]
    k_g = B._output_on(stream, target_k, (Bsz, L, hkv, n_keep, d), target_k.dtype)
    v_g = B._output_on(stream, target_k, k_g.shape, target_k.dtype)
    B.kv_compact(target_k, target_v, pc_idx, k_g, v_g, L * hkv, stream)
    out = speckv_compress(target_q, k_g, v_g, n_window, c_max, pool, stream=stream)
    return pc_scores, pc_idx, k_g, v_g, out


class PagedCache:
    """A paged KV cache on the device: k_pages, v_pages [L, n_pages, Hkv, page_rows,
    d], page_table int32 [n_seqs, max_pages], seq_lens int32 [n_seqs], page_refs
    int32 [n_pages].  The methods are the operators of the same names, and
    append; lists of sequences are int32 tensors.  write alone takes it that there
    was room: after a reserve that was refused it would go over rows the sequence
    holds, unless that reserve's result is given as `reserved`.  A layer at a
    time, tree_attention takes k_pages[l:l+1] and v_pages[l:l+1]."""

    def __init__(self, layers: int, n_pages: int, hkv: int, page_rows: int, head_dim: int, n_seqs: int, max_pages: int,
                 dtype=torch.bfloat16, device="cuda"):
        shape = (layers, n_pages, hkv, page_rows, head_dim)
        self.k_pages = torch.empty(shape, dtype=dtype, device=device)
        self.v_pages = torch.empty(shape, dtype=dtype, device=device)
        self.page_refs = torch.zeros(n_pages, dtype=torch.int32, device=device)
        self.page_table = torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device=device)
        self.seq_lens = torch.zeros(n_seqs, dtype=torch.int32, device=device)
        self.page_rows = page_rows

    @property
    def tensors(self):
        return self.k_pages, self.v_pages, self.page_refs, self.page_table, self.seq_lens

    def reserve(self, seqs, n_new, **kw):
        return B.kv_pages_reserve(*self.tensors, seqs, n_new, **kw)

    def write(self, k, v, seqs, **kw):
        B.kv_pages_write(k, v, *self.tensors, seqs, **kw)

    def append(self, k, v, seqs, counts, idx=None, units_per_idx: int = 1, stream=None):
        """Sequences seqs grow by counts int32 [n] rows and get them from k, v
        (reserve and write as one): returns reserve's result; unless it is 0
        nothing is changed."""
        result = self.reserve(seqs, counts, stream=stream)
        self.write(k, v, seqs, idx=idx, counts=counts, units_per_idx=units_per_idx, reserved=result, stream=stream)
        return result

    def compact(self, src, dst, idx, **kw):
        return B.kv_pages_compact(*self.tensors, src, dst, idx, **kw)

    def fork(self, src, dst, **kw):
        return B.kv_pages_fork(*self.tensors[2:], src, dst, page_rows=self.page_rows, **kw)

    def free(self, seqs, **kw):
        B.kv_pages_free(*self.tensors[2:], seqs, page_rows=self.page_rows, **kw)

    def attend(self, q, k_tree=None, v_tree=None, **kw):
        return B.tree_attention(q, self.k_pages, self.v_pages, self.page_table, self.seq_lens, k_tree, v_tree, **kw)


def speckv_compress_pages(q, k, v, n_window: int, c_max: int, cache: PagedCache, seqs, pool: int = 7,
                          scale: float = 1.0, stream=None, pool_mode: int = B.SPK_POOL_MAX):
    """SpecKV on every unit, with the kept rows written into the pages of
    sequences seqs int32 [B] (behind what they hold): returns (scores, idx,
    result); result as kv_pages_reserve's: unless it is 0 the cache is as it was."""
    Bsz, L, hkv, n_in, d = k.shape
    pages = cache.k_pages
    if v.shape != k.shape or (L, hkv, d) != (pages.shape[0], pages.shape[2], pages.shape[4]) or k.dtype != pages.dtype:
        raise ValueError(f"k and v are [B, L, Hkv, n_in, d] with the cache's L, Hkv, d and type, not {tuple(k.shape)}, "
                         f"{tuple(v.shape)}")
    if seqs.numel() != Bsz:
        raise ValueError(f"seqs names {seqs.numel()} sequences for a batch of {Bsz}")
    n_pre = n_in - n_window
    keep = min(c_max, n_pre) + n_window
    units = Bsz * L * hkv
    scores = B._output_on(stream, q, (units, n_pre), torch.float32)
    idx = B._output_on(stream, q, (units, keep), torch.int32)
    B.speckv_score(q, k, n_window, scores, None, None, scale, stream)
    B.topk_select(scores, c_max, n_window, idx, pool, None, None, stream, pool_mode)
    with torch.cuda.stream(B._stream_object(stream, q.device)):
        n_new = torch.full_like(seqs, keep)
    return scores, idx, cache.append(k, v, seqs, n_new, idx=idx, stream=stream)
