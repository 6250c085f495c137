"""MI355X (gfx950) lightning indexer + top-k token selector.

Thin Python binding over libdsaidx.so (include/dsaidx.h).  Every step of the
computation runs in the library's HIP kernels; this module only checks
tensor shapes, allocates outputs and workspace with torch on the inputs'
device, and passes pointers and the current HIP stream.

    indexer_prefill(q, k, w, topk, q_scale=None, k_scale=None, want_scores=False)
    indexer_decode_paged(q, w, k_cache, k_scale, block_table, context_lens, topk, max_context_len=None)
    topk_select(scores, topk, row_len=None)
    cache_append_rope(kv, seq_ids, positions, block_table, latent_cache, cos_sin, index_k=None, ...)
    latent_attention_topk(q, latent_cache, block_table, topk_idx, v_dim, scale, ...)
    latent_attention_shared(q, latent_cache, prefix_table, prefix_len, block_table, context_lens, v_dim, scale, ...)
    kv_append_rope(k, v, seq_ids, positions, block_table, k_cache, v_cache, cos_sin=None, ...)
    prompt_attention(q, k, v, cu_seqlens, scale, want_lse=False)
    kv_attention_decode(q, k_cache, v_cache, block_table, context_lens, scale, topk_idx=None, ...)

Input formats: fp32 tensors; bf16 as torch.bfloat16 or int16/uint16 bit
patterns; OCP FP8 E4M3 as torch.float8_e4m3fn or uint8 codes with fp32
per-row scales.
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad as _forward_ad

from . import _lib

F32, BF16, FP8_E4M3 = 0, 1, 2

__all__ = ["indexer_prefill", "indexer_prefill_noalloc", "indexer_decode_paged", "topk_select", "kcache_append", "topk_gather",
           "topk_gather_layers",
           "prefill_chunk_paged", "prefill_chunk_varlen",
           "cache_append_rope", "latent_attention_topk", "latent_attention_shared", "latent_topk_workspace_bytes",
           "latent_shared_workspace_bytes", "kv_append_rope", "prompt_attention", "kv_attention_decode",
           "kv_decode_workspace_bytes", "dtype_code", "F32", "BF16", "FP8_E4M3"]


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype in (torch.bfloat16, torch.int16, torch.uint16):
        return BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return FP8_E4M3
    raise TypeError(f"unsupported input dtype {t.dtype}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dev(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need(t, name: str, *dtypes) -> None:
    """Index and table tensors must be int32, weights and scales fp32: the
    library reads them as such, so any other element type would be read as
    garbage (an int64 block table as pairs of int32 page ids)."""
    if t is not None and t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")


_I32 = torch.int32
_F32 = torch.float32
_CODES = (torch.uint8, torch.float8_e4m3fn)


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# the same handle without the Python stream object (1.8 us a call) where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or _stream
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _workspace(nbytes: int, device) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def indexer_prefill(q, k, w, topk: int, q_scale=None, k_scale=None, want_scores: bool = False,
                    want_topk_score: bool = True):
    """Top-k causal history positions of every token of B sequences.

    q [B,L,H,D], k [B,L,D], w [B,L,H] fp32 (+ q_scale [B,L,H], k_scale [B,L]
    fp32 for fp8).  Returns (idx int32 [B,L,topk], score fp32 [B,L,topk] or
    None, scores fp32 [B,L,L] or None)."""
    lib = _lib.load()
    B, L, H, D = q.shape
    if tuple(k.shape) != (B, L, D) or tuple(w.shape) != (B, L, H):
        raise ValueError(f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)} w{tuple(w.shape)}")
    dt = dtype_code(q)
    if dtype_code(k) != dt:
        raise ValueError("q and k must share a format")
    _need(w, "w", _F32)
    _need(q_scale, "q_scale", _F32)
    _need(k_scale, "k_scale", _F32)
    for name, t in (("q", q), ("k", k), ("w", w), ("q_scale", q_scale), ("k_scale", k_scale)):
        if t is not None:
            _dev(t, name)
    dev = q.device
    idx = torch.empty((B, L, topk), dtype=torch.int32, device=dev)
    val = torch.empty((B, L, topk), dtype=torch.float32, device=dev) if want_topk_score else None
    scores = torch.empty((B, L, L), dtype=torch.float32, device=dev) if want_scores else None
    nws = lib.indexer_prefill_workspace_bytes(B, L, H, D, topk, dt, 1 if want_scores else 0)
    ws = _workspace(nws, dev)
    st = lib.indexer_prefill(_ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), dt, _ptr(w), B, L, H, D, topk,
                             _ptr(idx), _ptr(val), _ptr(scores), _ptr(ws), nws, _stream(dev))
    _lib.check(st, "indexer_prefill")
    return idx, val, scores


def indexer_prefill_noalloc(q, k, w, topk: int, q_scale=None, k_scale=None, want_scores: bool = False,
                            want_topk_score: bool = True, out=None):
    """indexer_prefill through the library entry point that allocates
    nothing (its scratch is a fixed device array inside the library).  The
    outputs are allocated here unless ``out`` = (idx, score or None, scores or
    None) gives them.  Returns the same triple as indexer_prefill."""
    lib = _lib.load()
    B, L, H, D = q.shape
    if tuple(k.shape) != (B, L, D) or tuple(w.shape) != (B, L, H):
        raise ValueError(f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)} w{tuple(w.shape)}")
    dt = dtype_code(q)
    if dtype_code(k) != dt:
        raise ValueError("q and k must share a format")
    _need(w, "w", _F32)
    _need(q_scale, "q_scale", _F32)
    _need(k_scale, "k_scale", _F32)
    for name, t in (("q", q), ("k", k), ("w", w), ("q_scale", q_scale), ("k_scale", k_scale)):
        if t is not None:
            _dev(t, name)
    dev = q.device
    if out is not None:
        idx, val, scores = out
        _need(idx, "idx", _I32)
        if tuple(idx.shape) != (B, L, topk) or (val is not None and tuple(val.shape) != (B, L, topk)) or \
                (scores is not None and tuple(scores.shape) != (B, L, L)):
            raise ValueError("output shapes do not match the call")
    else:
        idx = torch.empty((B, L, topk), dtype=torch.int32, device=dev)
        val = torch.empty((B, L, topk), dtype=torch.float32, device=dev) if want_topk_score else None
        scores = torch.empty((B, L, L), dtype=torch.float32, device=dev) if want_scores else None
    st = lib.indexer_prefill_noalloc(_ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), dt, _ptr(w), B, L, H, D, topk,
                                     _ptr(idx), _ptr(val), _ptr(scores), _stream(dev))
    _lib.check(st, "indexer_prefill_noalloc")
    return idx, val, scores


def indexer_decode_paged(q, w, k_cache, k_scale, block_table, context_lens, topk: int,
                         max_context_len: int | None = None, want_topk_score: bool = True,
                         workspace: torch.Tensor | None = None):
    """Top-k context positions of B decode queries over a paged fp8 cache.

    q [B,H,D] bf16, w [B,H] fp32, k_cache [P,page,D] fp8 codes, k_scale
    [P,page] fp32, block_table [B,max_pages] int32, context_lens [B] int32.
    ``max_context_len`` bounds context_lens (default: max_pages * page).
    Returns (idx int32 [B,topk], score fp32 [B,topk] or None)."""
    lib = _lib.load()
    B, H, D = q.shape
    P, page, Dk = k_cache.shape
    if Dk != D or tuple(k_scale.shape) != (P, page) or tuple(w.shape) != (B, H):
        raise ValueError("shape mismatch")
    if block_table.shape[0] != B or tuple(context_lens.shape) != (B,):
        raise ValueError("block_table / context_lens shape mismatch")
    _need(w, "w", _F32)
    _need(k_cache, "k_cache", *_CODES)
    _need(k_scale, "k_scale", _F32)
    _need(block_table, "block_table", _I32)
    _need(context_lens, "context_lens", _I32)
    for name, t in (("q", q), ("w", w), ("k_cache", k_cache), ("k_scale", k_scale),
                    ("block_table", block_table), ("context_lens", context_lens)):
        _dev(t, name)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    mpp = block_table.shape[1]
    mcl = mpp * page if max_context_len is None else int(max_context_len)
    dev = q.device
    idx = torch.empty((B, topk), dtype=torch.int32, device=dev)
    val = torch.empty((B, topk), dtype=torch.float32, device=dev) if want_topk_score else None
    nws = lib.indexer_decode_paged_workspace_bytes(B, mcl, H, D, topk)
    ws = workspace if workspace is not None and workspace.numel() >= nws else _workspace(nws, dev)
    st = lib.indexer_decode_paged(_ptr(q), dtype_code(q), _ptr(w), _ptr(k_cache), _ptr(k_scale),
                                  _ptr(block_table), mpp, _ptr(context_lens), mcl, B, H, D, page, P, topk,
                                  _ptr(idx), _ptr(val), _ptr(ws), nws, _stream(dev))
    _lib.check(st, "indexer_decode_paged")
    return idx, val


def decode_workspace_bytes(B: int, max_context_len: int, H: int, D: int, topk: int) -> int:
    return _lib.load().indexer_decode_paged_workspace_bytes(B, max_context_len, H, D, topk)


def topk_select(scores, topk: int, row_len=None, want_values: bool = True):
    """Top-k of each row of a [rows, cols] fp32 matrix (row r valid up to
    row_len[r]).  Returns (idx int32 [rows,topk], values fp32 or None)."""
    lib = _lib.load()
    if scores.dim() != 2 or scores.dtype != torch.float32:
        raise ValueError("scores must be a 2-D fp32 tensor")
    if scores.stride(1) != 1:
        raise ValueError("scores rows must be contiguous")
    rows, cols = scores.shape
    dev = scores.device
    if row_len is not None:
        _need(row_len, "row_len", _I32)
        _dev(row_len, "row_len")
        if tuple(row_len.shape) != (rows,):
            raise ValueError("row_len must hold one length per row")
    idx = torch.empty((rows, topk), dtype=torch.int32, device=dev)
    val = torch.empty((rows, topk), dtype=torch.float32, device=dev) if want_values else None
    nws = lib.topk_select_workspace_bytes(rows, cols, topk)
    ws = _workspace(nws, dev)
    st = lib.topk_select(_ptr(scores), rows, cols, scores.stride(0), _ptr(row_len), topk, _ptr(idx), _ptr(val),
                         _ptr(ws), nws, _stream(dev))
    _lib.check(st, "topk_select")
    return idx, val


def kcache_append(k, seq_ids, positions, block_table, k_cache, k_scale):
    """Quantise T new keys to FP8 and write them into the paged cache in place.

    k [T,D] bf16 or fp32, seq_ids [T] int32 (outside [0, B): skipped),
    positions [T] int32, block_table [B,max_pages] int32, k_cache [P,page,D]
    uint8 E4M3FN codes, k_scale [P,page] fp32.  Returns nothing: k_cache and
    k_scale are updated on the current stream."""
    lib = _lib.load()
    T, D = k.shape
    P, page, Dk = k_cache.shape
    if Dk != D or tuple(k_scale.shape) != (P, page):
        raise ValueError("k_cache / k_scale shape mismatch")
    if tuple(seq_ids.shape) != (T,) or tuple(positions.shape) != (T,):
        raise ValueError("seq_ids / positions must have one entry per key")
    if k_cache.dtype != torch.uint8 or k_scale.dtype != torch.float32:
        raise ValueError("k_cache must be uint8 codes and k_scale fp32")
    _need(seq_ids, "seq_ids", _I32)
    _need(positions, "positions", _I32)
    _need(block_table, "block_table", _I32)
    for name, t in (("k", k), ("seq_ids", seq_ids), ("positions", positions), ("block_table", block_table),
                    ("k_cache", k_cache), ("k_scale", k_scale)):
        _dev(t, name)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    B, mpp = block_table.shape
    st = lib.indexer_kcache_append(_ptr(k), dtype_code(k), _ptr(seq_ids), _ptr(positions), _ptr(block_table),
                                   B, mpp, _ptr(k_cache), _ptr(k_scale), P, T, D, page, _stream(k.device))
    _lib.check(st, "indexer_kcache_append")


def topk_gather(latent_cache, block_table, topk_idx):
    """Rows of a paged latent cache at each query's selected positions.

    latent_cache [P,page,E] (any element type; E * element size a multiple of
    16 bytes), block_table [B,max_pages] int32, topk_idx [B,K] int32 (-1 or
    outside the table: a zero row).  Returns out [B,K,E] of the cache's dtype."""
    lib = _lib.load()
    P, page, E = latent_cache.shape
    B, K = topk_idx.shape
    if block_table.shape[0] != B or topk_idx.dtype != torch.int32 or block_table.dtype != torch.int32:
        raise ValueError("block_table [B, max_pages] and topk_idx [B, K] must be int32 with matching B")
    for name, t in (("latent_cache", latent_cache), ("block_table", block_table), ("topk_idx", topk_idx)):
        _dev(t, name)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    out = torch.empty((B, K, E), dtype=latent_cache.dtype, device=latent_cache.device)
    st = lib.indexer_topk_gather(_ptr(latent_cache), E * latent_cache.element_size(), _ptr(block_table),
                                 block_table.shape[1], P, page, _ptr(topk_idx), B, K, _ptr(out),
                                 _stream(latent_cache.device))
    _lib.check(st, "indexer_topk_gather")
    return out


def topk_gather_layers(latent_caches, block_table, topk_idx, outs=None):
    """Index Share: one selection gathered from several layers' latent
    caches in one launch.  latent_caches: a sequence of [P,page,E] tensors of
    one shape and dtype (at most 64); block_table, topk_idx as topk_gather.
    Returns a list of [B,K,E] tensors, one per layer (or fills `outs`)."""
    import ctypes

    lib = _lib.load()
    caches = list(latent_caches)
    if not caches:
        raise ValueError("latent_caches is empty")
    P, page, E = caches[0].shape
    for i, c in enumerate(caches):
        if c.shape != caches[0].shape or c.dtype != caches[0].dtype:
            raise ValueError(f"latent_caches[{i}] differs in shape or dtype from latent_caches[0]")
        _dev(c, f"latent_caches[{i}]")
    B, K = topk_idx.shape
    _need(block_table, "block_table", _I32)
    _need(topk_idx, "topk_idx", _I32)
    for name, t in (("block_table", block_table), ("topk_idx", topk_idx)):
        _dev(t, name)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages] with the B of topk_idx")
    if outs is None:
        outs = [torch.empty((B, K, E), dtype=caches[0].dtype, device=caches[0].device) for _ in caches]
    else:
        outs = list(outs)
        if len(outs) != len(caches):
            raise ValueError("one output per layer")
        for i, o in enumerate(outs):
            if o.shape != (B, K, E) or o.dtype != caches[0].dtype:
                raise ValueError(f"outs[{i}] must be [B, K, E] of the caches' dtype")
            _dev(o, f"outs[{i}]")
    n = len(caches)
    cp = (ctypes.c_void_p * n)(*[c.data_ptr() for c in caches])
    op = (ctypes.c_void_p * n)(*[o.data_ptr() for o in outs])
    st = lib.indexer_topk_gather_layers(cp, op, n, E * caches[0].element_size(), _ptr(block_table),
                                        block_table.shape[1], P, page, _ptr(topk_idx), B, K,
                                        _stream(caches[0].device))
    _lib.check(st, "indexer_topk_gather_layers")
    return outs


def probe_mfma(kind: int, blocks: int, iters: int, device="cuda"):
    """Measurement probe: blocks x 4 waves x iters x 8 MFMAs of one shape
    (0: fp8 16x16x128 scaled, 1: bf16 16x16x32, 2: f16 16x16x32).  Returns
    the (meaningless) output tensor; time the call with events."""
    out = torch.empty(blocks * 256, dtype=torch.float32, device=device)
    _lib.check(_lib.load().dsaidx_probe_mfma(kind, blocks, iters, _ptr(out), _stream(out.device)),
               "dsaidx_probe_mfma")
    return out


def probe_page_read(k_cache, k_scale, page_ids, blocks: int, out=None):
    """Measurement probe: reads the pages page_ids of a paged fp8 key cache
    (8448 bytes each) with the decode scan's load layout."""
    _need(k_cache, "k_cache", *_CODES)
    _need(k_scale, "k_scale", _F32)
    _need(page_ids, "page_ids", _I32)
    for name, t in (("k_cache", k_cache), ("k_scale", k_scale), ("page_ids", page_ids)):
        _dev(t, name)
    if out is None:
        out = torch.empty(blocks * 256, dtype=torch.float32, device=k_cache.device)
    _lib.check(_lib.load().dsaidx_probe_page_read(_ptr(k_cache), _ptr(k_scale), _ptr(page_ids), page_ids.numel(),
                                                  blocks, _ptr(out), _stream(k_cache.device)),
               "dsaidx_probe_page_read")
    return out


def prefill_chunk_varlen(q, q_scale, w, cu_seqlens_q, q_start, k_cache, k_scale, block_table, topk: int,
                         max_kv_len: int, want_topk_score: bool = True, workspace: torch.Tensor | None = None):
    """Top-k of the query rows of B sequences' chunks (packed one after
    another) against the paged fp8 key cache: row cu_seqlens_q[b] + i is
    position q_start[b] + i of sequence b and sees keys 0 .. that position.

    q [T,H,D] fp8 codes (uint8) with q_scale [T,H] fp32, or bf16 with
    q_scale None; w [T,H] fp32,
    cu_seqlens_q [B+1] int32 (device), q_start [B] int32 (device), k_cache
    [P,page,D] uint8, k_scale [P,page] fp32, block_table [B,max_pages] int32;
    ``max_kv_len`` bounds q_start[b] + rows of b (host value).  Returns (idx
    int32 [T,topk] of absolute positions, score fp32 [T,topk] or None)."""
    lib = _lib.load()
    T, H, D = q.shape
    P, page, Dk = k_cache.shape
    B = q_start.shape[0]
    if Dk != D or tuple(k_scale.shape) != (P, page) or tuple(w.shape) != (T, H):
        raise ValueError("shape mismatch")
    fp8_q = dtype_code(q) == FP8_E4M3
    if fp8_q != (q_scale is not None):
        raise ValueError("q_scale [T, H] goes with fp8 queries, None with bf16 queries")
    if q_scale is not None and tuple(q_scale.shape) != (T, H):
        raise ValueError("q_scale must be [T, H]")
    if tuple(cu_seqlens_q.shape) != (B + 1,) or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("cu_seqlens_q [B+1], q_start [B] and block_table [B, max_pages] must agree on B")
    _need(q, "q", *_CODES, torch.bfloat16, torch.int16, torch.uint16)
    _need(q_scale, "q_scale", _F32)
    _need(w, "w", _F32)
    _need(k_cache, "k_cache", *_CODES)
    _need(k_scale, "k_scale", _F32)
    _need(block_table, "block_table", _I32)
    _need(cu_seqlens_q, "cu_seqlens_q", _I32)
    _need(q_start, "q_start", _I32)
    for name, t in (("q", q), ("q_scale", q_scale), ("w", w), ("cu_seqlens_q", cu_seqlens_q), ("q_start", q_start),
                    ("k_cache", k_cache), ("k_scale", k_scale), ("block_table", block_table)):
        if t is not None:
            _dev(t, name)
    dev = q.device
    idx = torch.empty((T, topk), dtype=torch.int32, device=dev)
    val = torch.empty((T, topk), dtype=torch.float32, device=dev) if want_topk_score else None
    nws = lib.indexer_prefill_chunk_paged_workspace_bytes(B, T, int(max_kv_len), dtype_code(q))
    ws = workspace if workspace is not None and workspace.numel() >= nws else _workspace(nws, dev)
    st = lib.indexer_prefill_chunk_paged(_ptr(q), _ptr(q_scale), dtype_code(q), _ptr(w), _ptr(cu_seqlens_q),
                                         _ptr(q_start), _ptr(k_cache), _ptr(k_scale), _ptr(block_table),
                                         block_table.shape[1], P, B, T, int(max_kv_len), H, D, page, topk,
                                         _ptr(idx), _ptr(val), _ptr(ws), nws, _stream(dev))
    _lib.check(st, "indexer_prefill_chunk_paged")
    return idx, val


def prefill_chunk_paged(q, q_scale, w, k_cache, k_scale, block_table, q0: int, topk: int,
                        want_topk_score: bool = True, workspace: torch.Tensor | None = None):
    """Top-k of a chunk of Lq query tokens per sequence, all at positions q0
    .. q0+Lq-1, against a paged fp8 key cache that holds keys 0 .. q0+Lq-1
    (prefill_chunk_varlen with equal chunks).

    q [B,Lq,H,D] fp8 codes (uint8) with q_scale [B,Lq,H] fp32, or bf16 with
    q_scale None; w [B,Lq,H] fp32, k_cache [P,page,D] uint8, k_scale [P,page]
    fp32, block_table [B,max_pages] int32.  Returns (idx int32 [B,Lq,topk] of
    absolute positions, score fp32 or None)."""
    B, Lq, H, D = q.shape
    if tuple(w.shape) != (B, Lq, H) or block_table.shape[0] != B:
        raise ValueError("w / block_table shape mismatch")
    if q_scale is not None and tuple(q_scale.shape) != (B, Lq, H):
        raise ValueError("q_scale must be [B, Lq, H]")
    dev = q.device
    cu = torch.arange(0, (B + 1) * Lq, Lq, dtype=torch.int32, device=dev)
    qs = torch.full((B,), int(q0), dtype=torch.int32, device=dev)
    qsc = None if q_scale is None else q_scale.reshape(B * Lq, H)
    idx, val = prefill_chunk_varlen(q.reshape(B * Lq, H, D), qsc, w.reshape(B * Lq, H), cu, qs,
                                    k_cache, k_scale, block_table, topk, int(q0) + Lq,
                                    want_topk_score=want_topk_score, workspace=workspace)
    return idx.view(B, Lq, topk), None if val is None else val.view(B, Lq, topk)


def _all(index: int, checks) -> None:
    """(name, tensor or None, element types): each tensor of one of its types,
    contiguous, on GPU `index`."""
    for _, t, dtypes in checks:
        if t is not None and (t.dtype not in dtypes or t.get_device() != index or not t.is_contiguous()):
            break
    else:
        if index >= 0:
            return
    for name, t, dtypes in checks:
        _need(t, name, *dtypes)
    for name, t, _ in checks:
        if t is not None:
            _dev(t, name)
            if t.get_device() != index:
                raise ValueError(f"{name} must be on device {index}, the device of the other tensors")


def _rows(t, name: str) -> int:
    """Row stride (elements) of a 2-D device tensor whose rows are contiguous."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    s = t.stride()
    if len(s) != 2 or (s[1] != 1 and t.shape[1] != 1):
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    return s[0]


def _dual_level() -> bool:
    """Whether this is within a forward_ad.dual_level(), outside of which no tensor has a tangent."""
    return getattr(_forward_ad, "_current_level", 0) >= 0


def _derivatives() -> bool:
    return torch.is_grad_enabled() or _dual_level()


def _inference_only(where: str, *tensors) -> None:
    """Refuses inputs with a derivative, which the call would drop: a gradient (where gradients are enabled) or a
    tangent (which no_grad does not switch off)."""
    grad, dual = torch.is_grad_enabled(), _dual_level()
    for t in tensors:
        if t is not None and grad and t.requires_grad:
            raise ValueError(f"{where} has no backward: call it under torch.no_grad() or detach its inputs")
        if t is not None and dual and _forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError(f"{where} has no forward derivative: call it with the primals of its dual inputs")


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_NEW = _BF16 + (torch.float32,)
_LATENT = _BF16 + _CODES
_FLOATS = (torch.float32,)
_INTS = (torch.int32,)


def cache_append_rope(kv, seq_ids, positions, block_table, latent_cache, cos_sin, latent_scale=None,
                      kv_interleaved: bool = True, index_k=None, k_cache=None, k_scale=None,
                      index_interleaved: bool = False) -> None:
    """Rotates T new tokens' latent rows and index keys by their positions and
    writes them into the two paged caches in place, in one launch.

    kv [T,E] bf16 or fp32 (rows may be strided), its last R columns rotated;
    cos_sin [rope_len,R] fp32 (R/2 cosines, then R/2 sines, of each position);
    seq_ids, positions [T] int32 (a token outside the table, rope_len or the
    pool is skipped); block_table [B,max_pages] int32; latent_cache [P,page,E]
    bf16, or uint8 / float8_e4m3fn codes with latent_scale [P,page] fp32.
    index_k [T,D] (kv's type, its first R columns rotated) goes to k_cache
    [P,page,D] codes and k_scale [P,page] fp32 as kcache_append writes them;
    all three None: latent rows only.  kv_interleaved, index_interleaved: pair
    i is columns (2i, 2i+1), else (i, i + R/2).  Returns nothing."""
    lib = _lib.load()
    index = kv.get_device()
    dtype = kv.dtype
    if dtype not in _NEW:
        _need(kv, "kv", *_NEW)
    kv_stride = _rows(kv, "kv")
    T, E = kv.shape
    _all(index, (("latent_cache", latent_cache, _LATENT), ("latent_scale", latent_scale, _FLOATS),
                 ("cos_sin", cos_sin, _FLOATS), ("seq_ids", seq_ids, _INTS), ("positions", positions, _INTS),
                 ("block_table", block_table, _INTS), ("k_cache", k_cache, _CODES), ("k_scale", k_scale, _FLOATS)))
    shape = latent_cache.shape
    if len(shape) != 3 or shape[2] != E:
        raise ValueError("latent_cache must be [P, page, E] with the E of kv")
    P, page, _ = shape
    fp8 = latent_cache.dtype in _CODES
    if fp8 != (latent_scale is not None) or (fp8 and latent_scale.shape != (P, page)):
        raise ValueError("latent_scale [P, page] goes with fp8 latent rows, None with bf16 rows")
    if cos_sin.dim() != 2 or block_table.dim() != 2:
        raise ValueError("cos_sin must be [rope_len, R] and block_table [B, max_pages]")
    if seq_ids.shape != (T,) or positions.shape != (T,):
        raise ValueError("seq_ids / positions must have one entry per token")
    index_stride, D = 0, 128
    if (index_k is None) != (k_cache is None) or (index_k is None) != (k_scale is None):
        raise ValueError("index_k, k_cache and k_scale go together")
    if index_k is not None:
        index_stride = _rows(index_k, "index_k")
        n, D = index_k.shape
        if index_k.dtype != dtype or n != T or index_k.get_device() != index:
            raise ValueError("index_k must be [T, D] of kv's type, on its device")
        if k_cache.shape != (P, page, D) or k_scale.shape != (P, page):
            raise ValueError("k_cache [P, page, D] / k_scale [P, page] shape mismatch")
    _inference_only("cache_append_rope", kv, index_k, cos_sin, latent_cache, latent_scale, k_scale)
    B, max_pages = block_table.shape
    rope_len, R = cos_sin.shape
    if _current_device() != index:
        with torch.cuda.device(index):
            return cache_append_rope(kv, seq_ids, positions, block_table, latent_cache, cos_sin, latent_scale,
                                     kv_interleaved, index_k, k_cache, k_scale, index_interleaved)
    st = lib.indexer_cache_append_rope(kv.data_ptr(), kv_stride, 1 if kv_interleaved else 0, _ptr(index_k),
                                       index_stride, 1 if index_interleaved else 0,
                                       F32 if dtype == torch.float32 else BF16, cos_sin.data_ptr(), rope_len, R,
                                       seq_ids.data_ptr(), positions.data_ptr(), block_table.data_ptr(), B, max_pages,
                                       latent_cache.data_ptr(), _ptr(latent_scale), FP8_E4M3 if fp8 else BF16,
                                       _ptr(k_cache), _ptr(k_scale), P, T, E, D, page, _raw_stream(index))
    if st:
        _lib.check(st, "indexer_cache_append_rope")


def _latent_inputs(q, latent_cache, latent_scale, block_table, where: str, *others):
    """Checks that the latent-attention calls share; returns (P, page, dtype code of the rows)."""
    _all(q.get_device(), (("q", q, _BF16), ("latent_cache", latent_cache, _LATENT),
                          ("latent_scale", latent_scale, _FLOATS), ("block_table", block_table, _INTS), *others))
    shape = latent_cache.shape
    if q.dim() != 3 or len(shape) != 3 or shape[2] != q.shape[2]:
        raise ValueError("q must be [rows, H, E] and latent_cache [P, page, E]")
    P, page, _ = shape
    fp8 = latent_cache.dtype in _CODES
    if fp8 != (latent_scale is not None) or (fp8 and latent_scale.shape != (P, page)):
        raise ValueError("latent_scale [P, page] goes with fp8 latent rows, None with bf16 rows")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    _inference_only(where, q, latent_cache, latent_scale)
    return P, page, FP8_E4M3 if fp8 else BF16


def _scratch(workspace, nbytes: int, q):
    """The caller's workspace where it is one (enough bytes, on q's device), else a new one; None where none is needed."""
    if nbytes == 0:
        return None
    if workspace is not None:
        if workspace.get_device() != q.get_device() or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {q.device}")
        if workspace.numel() * workspace.element_size() >= nbytes:
            return workspace
    return q.new_empty(nbytes, dtype=torch.uint8)


def latent_topk_workspace_bytes(T: int, H: int, E: int, v_dim: int, topk: int, fp8: bool = False) -> int:
    return _lib.load().indexer_latent_attention_topk_workspace_bytes(T, H, E, v_dim, topk, FP8_E4M3 if fp8 else BF16)


def latent_shared_workspace_bytes(B: int, H: int, E: int, v_dim: int, prefix_len: int, max_context_len: int,
                                  fp8: bool = False) -> int:
    return _lib.load().indexer_latent_attention_shared_workspace_bytes(B, H, E, v_dim, prefix_len, max_context_len,
                                                                       FP8_E4M3 if fp8 else BF16)


def latent_attention_topk(q, latent_cache, block_table, topk_idx, v_dim: int, scale: float, latent_scale=None,
                          seq_ids=None, want_lse: bool = False, workspace: torch.Tensor | None = None):
    """Attention of every head over the latent rows at each query's selected
    positions, read in place (no gathered copy).

    q [T,H,E] bf16, latent_cache [P,page,E] bf16, or uint8 / float8_e4m3fn
    codes with latent_scale [P,page] fp32; the first v_dim columns of a row are
    its value.  block_table [B,max_pages] int32; topk_idx [T,K] int32 positions
    (-1, or outside the table: no row); seq_ids [T] int32 gives each query's
    row of the table (outside [0, B): no rows), None: query t uses row t.
    ``workspace``: the caller's scratch of latent_topk_workspace_bytes, not
    shared by calls in flight (default: a new one each call).
    Returns (out bf16 [T,H,v_dim], lse fp32 [T,H] or None); a query without a
    row gives zeros and -inf."""
    lib = _lib.load()
    P, page, dt = _latent_inputs(q, latent_cache, latent_scale, block_table, "latent_attention_topk",
                                 ("topk_idx", topk_idx, _INTS), ("seq_ids", seq_ids, _INTS))
    T, H, E = q.shape
    if topk_idx.dim() != 2 or topk_idx.shape[0] != T:
        raise ValueError("topk_idx must be [T, K]")
    if seq_ids is not None and seq_ids.shape != (T,):
        raise ValueError("seq_ids must have one entry per query")
    B, max_pages = block_table.shape
    if seq_ids is None and B != T:
        raise ValueError("block_table must have one row per query (or give seq_ids)")
    K, index = topk_idx.shape[1], q.get_device()
    if _current_device() != index:
        with torch.cuda.device(index):
            return latent_attention_topk(q, latent_cache, block_table, topk_idx, v_dim, scale, latent_scale, seq_ids,
                                         want_lse, workspace)
    out = q.new_empty((T, H, v_dim), dtype=torch.bfloat16)
    lse = q.new_empty((T, H), dtype=torch.float32) if want_lse else None
    nws = lib.indexer_latent_attention_topk_workspace_bytes(T, H, E, v_dim, K, dt)
    ws = _scratch(workspace, nws, q)
    st = lib.indexer_latent_attention_topk(q.data_ptr(), BF16, latent_cache.data_ptr(), _ptr(latent_scale), dt,
                                           block_table.data_ptr(), max_pages, P, topk_idx.data_ptr(), _ptr(seq_ids),
                                           B or 1, T, H, E, v_dim, page, K, scale, out.data_ptr(), _ptr(lse),
                                           _ptr(ws), nws, _raw_stream(index))
    if st:
        _lib.check(st, "indexer_latent_attention_topk")
    return out, lse


def latent_attention_shared(q, latent_cache, prefix_table, prefix_len: int, block_table, context_lens, v_dim: int,
                            scale: float, max_context_len: int | None = None, latent_scale=None,
                            want_lse: bool = False, workspace: torch.Tensor | None = None):
    """One decode step of B queries over a prefix that all of them share, read
    once for each block of up to 128 query rows, and each sequence's own
    positions behind it.

    q [B,H,E] bf16, latent_cache and latent_scale as latent_attention_topk;
    prefix_table [n] int32 page ids of the prefix's first ``prefix_len``
    positions (None when that is 0); block_table [B,max_pages] int32 and
    context_lens [B] int32: the sequences' own pages and lengths.
    ``max_context_len`` bounds context_lens (default: max_pages * page); the work
    is cut for contexts of that length, so a bound near the longest is faster.
    ``workspace``: the caller's scratch of latent_shared_workspace_bytes, not
    shared by calls in flight (default: a new one each call).
    Returns (out bf16 [B,H,v_dim], lse fp32 [B,H] or None); a query without a
    position gives zeros and -inf."""
    lib = _lib.load()
    P, page, dt = _latent_inputs(q, latent_cache, latent_scale, block_table, "latent_attention_shared",
                                 ("prefix_table", prefix_table, _INTS), ("context_lens", context_lens, _INTS))
    B, H, E = q.shape
    if block_table.shape[0] != B or context_lens.shape != (B,):
        raise ValueError("block_table / context_lens shape mismatch")
    if prefix_table is not None and prefix_table.dim() != 1:
        raise ValueError("prefix_table must be one-dimensional")
    max_pages = block_table.shape[1]
    mcl = max_pages * page if max_context_len is None else int(max_context_len)
    if prefix_len >> 31 or mcl >> 31:
        raise ValueError("prefix_len and max_context_len must be in [0, 2^31)")
    index = q.get_device()
    if _current_device() != index:
        with torch.cuda.device(index):
            return latent_attention_shared(q, latent_cache, prefix_table, prefix_len, block_table, context_lens,
                                           v_dim, scale, max_context_len, latent_scale, want_lse, workspace)
    out = q.new_empty((B, H, v_dim), dtype=torch.bfloat16)
    lse = q.new_empty((B, H), dtype=torch.float32) if want_lse else None
    nws = lib.indexer_latent_attention_shared_workspace_bytes(B, H, E, v_dim, prefix_len, mcl, dt)
    ws = _scratch(workspace, nws, q)
    st = lib.indexer_latent_attention_shared(q.data_ptr(), BF16, latent_cache.data_ptr(), _ptr(latent_scale), dt,
                                             _ptr(prefix_table), 0 if prefix_table is None else prefix_table.shape[0],
                                             prefix_len, block_table.data_ptr(), max_pages, P,
                                             context_lens.data_ptr(), mcl, B, H, E, v_dim, page, scale, out.data_ptr(),
                                             _ptr(lse), _ptr(ws), nws, _raw_stream(index))
    if st:
        _lib.check(st, "indexer_latent_attention_shared")
    return out, lse


def _heads(t, name: str, index: int, dtypes):
    """Token and head stride (elements) of a [T, heads, columns] tensor on GPU `index` whose rows are contiguous."""
    if t.dtype not in dtypes:
        _need(t, name, *dtypes)
    if t.get_device() != index or index < 0:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        raise ValueError(f"{name} must be on device {index}, the device of the other tensors")
    s = t.stride()
    if len(s) != 3 or (s[2] != 1 and t.shape[2] != 1):
        raise ValueError(f"{name} must be [tokens, heads, columns] with contiguous rows")
    return s[0], s[1]


def _kv_caches(index: int, k_cache, v_cache, k_scale, v_scale, G: int, D: int):
    """Checks of the paged key and value caches; returns (P, page, dtype code)."""
    shape, dtype = k_cache.shape, k_cache.dtype
    if index < 0 or dtype not in _LATENT or v_cache.dtype not in _LATENT or k_cache.get_device() != index or \
            v_cache.get_device() != index or not k_cache.is_contiguous() or not v_cache.is_contiguous() or \
            k_scale is not None or v_scale is not None:
        _all(index, (("k_cache", k_cache, _LATENT), ("v_cache", v_cache, _LATENT), ("k_scale", k_scale, _FLOATS),
                     ("v_scale", v_scale, _FLOATS)))
    if len(shape) != 4 or shape[1] != G or shape[3] != D or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be [P, G, page, D] with the G and D of the other tensors")
    fp8 = dtype in _CODES
    if (v_cache.dtype in _CODES) != fp8:
        raise ValueError("k_cache and v_cache must both be bf16 or both fp8")
    if fp8 or k_scale is not None or v_scale is not None:
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if fp8 != (s is not None) or (fp8 and s.shape != shape[:3]):
                raise ValueError(f"{name} [P, G, page] goes with fp8 caches, None with bf16 ones")
    return shape[0], shape[2], FP8_E4M3 if fp8 else BF16


def _indices(index: int, checks) -> None:
    """(name, int32 tensor), contiguous, on GPU `index`."""
    for _, t in checks:
        if t.dtype is not _I32 or t.get_device() != index or not t.is_contiguous():
            _all(index, [(name, x, _INTS) for name, x in checks])


def kv_append_rope(k, v, seq_ids, positions, block_table, k_cache, v_cache, cos_sin=None, k_scale=None, v_scale=None,
                   interleaved: bool = False) -> None:
    """Writes T new tokens' keys, rotated by their positions, and values into
    paged caches with G heads of their own, in place, in one launch.

    k, v [T,G,D] bf16 or fp32 (tokens and heads may be strided); cos_sin
    [rope_len,R] fp32 (R/2 cosines, then R/2 sines, of each position) turns the
    first R columns of every key, None: no rotation; seq_ids, positions [T] int32
    (a token outside the table, rope_len or the pool is skipped); block_table
    [B,max_pages] int32; k_cache, v_cache [P,G,page,D] bf16, or uint8 /
    float8_e4m3fn codes with k_scale, v_scale [P,G,page] fp32.  interleaved: pair
    i is columns (2i, 2i+1), else (i, i + R/2).  Returns nothing."""
    lib = _lib.load()
    index = k.get_device()
    ks, kh = _heads(k, "k", index, _NEW)
    vs, vh = _heads(v, "v", index, _NEW)
    T, G, D = k.shape
    if v.shape != k.shape or (v.dtype is _F32) != (k.dtype is _F32):
        raise ValueError("k and v must be [T, G, D] of one type")
    P, page, dt = _kv_caches(index, k_cache, v_cache, k_scale, v_scale, G, D)
    _indices(index, (("seq_ids", seq_ids), ("positions", positions), ("block_table", block_table)))
    if cos_sin is not None and (cos_sin.dtype is not _F32 or cos_sin.get_device() != index or
                                not cos_sin.is_contiguous()):
        _all(index, (("cos_sin", cos_sin, _FLOATS),))
    if block_table.dim() != 2 or (cos_sin is not None and (cos_sin.dim() != 2 or cos_sin.numel() == 0)):
        # (a table without an entry has no address: it would read as None, no rotation)
        raise ValueError("cos_sin must be [rope_len, R], neither of them 0, and block_table [B, max_pages]")
    if seq_ids.shape != (T,) or positions.shape != (T,):
        raise ValueError("seq_ids / positions must have one entry per token")
    if _derivatives():
        _inference_only("kv_append_rope", k, v, cos_sin, k_cache, v_cache, k_scale, v_scale)
    B, max_pages = block_table.shape
    rope_len, R = (0, 0) if cos_sin is None else cos_sin.shape
    if _current_device() != index:
        with torch.cuda.device(index):
            return kv_append_rope(k, v, seq_ids, positions, block_table, k_cache, v_cache, cos_sin, k_scale, v_scale,
                                  interleaved)
    st = lib.indexer_kv_append_rope(k.data_ptr(), ks, kh, v.data_ptr(), vs, vh,
                                    F32 if k.dtype is _F32 else BF16, _ptr(cos_sin), rope_len, R,
                                    1 if interleaved else 0, seq_ids.data_ptr(), positions.data_ptr(),
                                    block_table.data_ptr(), B, max_pages, k_cache.data_ptr(), _ptr(k_scale),
                                    v_cache.data_ptr(), _ptr(v_scale), dt, P, T, G, D, page, _raw_stream(index))
    if st:
        _lib.check(st, "indexer_kv_append_rope")


def prompt_attention(q, k, v, cu_seqlens, scale: float, want_lse: bool = False):
    """Causal attention over whole prompts, packed one after another, with
    grouped heads: row i of a sequence attends over its rows 0 .. i, query head h
    over key/value head h // (H / G).

    q [T,H,D], k [T,G,D], v [T,G,V] bf16 (tokens and heads may be strided);
    cu_seqlens [B+1] int32 (device): sequence b is rows cu_seqlens[b] ..
    cu_seqlens[b+1]-1.  Returns (out bf16 [T,H,V], lse fp32 [T,H] or None); rows
    behind the last sequence give zeros and -inf."""
    lib = _lib.load()
    index = q.get_device()
    qs, qh = _heads(q, "q", index, _BF16)
    ks, kh = _heads(k, "k", index, _BF16)
    vs, vh = _heads(v, "v", index, _BF16)
    _indices(index, (("cu_seqlens", cu_seqlens),))
    T, H, D = q.shape
    _, G, V = v.shape
    if k.shape != (T, G, D) or v.shape[0] != T:
        raise ValueError("q must be [T, H, D], k [T, G, D] and v [T, G, V]")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must be [B + 1] with B >= 1")
    if _derivatives():
        _inference_only("prompt_attention", q, k, v)
    if _current_device() != index:
        with torch.cuda.device(index):
            return prompt_attention(q, k, v, cu_seqlens, scale, want_lse)
    out = q.new_empty((T, H, V), dtype=torch.bfloat16)
    lse = q.new_empty((T, H), dtype=torch.float32) if want_lse else None
    st = lib.indexer_prompt_attention(q.data_ptr(), qs, qh, k.data_ptr(), ks, kh, v.data_ptr(), vs, vh, BF16,
                                      cu_seqlens.data_ptr(), cu_seqlens.shape[0] - 1, T, H, G, D, V, scale,
                                      out.data_ptr(), _ptr(lse), _raw_stream(index))
    if st:
        _lib.check(st, "indexer_prompt_attention")
    return out, lse


def kv_decode_workspace_bytes(B: int, H: int, G: int, D: int, max_context_len: int, topk: int = 0,
                              fp8: bool = False) -> int:
    return _lib.load().indexer_kv_attention_decode_workspace_bytes(B, H, G, D, max_context_len, topk,
                                                                   FP8_E4M3 if fp8 else BF16)


def kv_attention_decode(q, k_cache, v_cache, block_table, context_lens, scale: float, topk_idx=None,
                        max_context_len: int | None = None, k_scale=None, v_scale=None, want_lse: bool = False,
                        workspace: torch.Tensor | None = None):
    """One decode step over paged caches with G key/value heads: the new token of
    each of B sequences attends over its whole context, or over the positions
    selected for it; query head h reads key/value head h // (H / G).

    q [B,H,D] bf16, contiguous; k_cache, v_cache [P,G,page,D] bf16, or uint8 /
    float8_e4m3fn codes with k_scale, v_scale [P,G,page] fp32, as kv_append_rope
    writes them; block_table [B,max_pages] int32; context_lens [B] int32; topk_idx
    [B,K] int32 positions (-1, or outside the context: no row), None: every position.
    ``max_context_len`` bounds context_lens (default: max_pages * page); the work,
    and the workspace, are cut for contexts of that length, so a bound near the
    longest is faster (128 contexts of 300: 28 us, with a bound of 131072 112).
    ``workspace``: the caller's scratch of kv_decode_workspace_bytes, not shared
    by calls in flight (default: a new one each call).
    Returns (out bf16 [B,H,D], lse fp32 [B,H] or None); a query without a position
    gives zeros and -inf."""
    lib = _lib.load()
    index = q.get_device()
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [B, H, D] and the caches [P, G, page, D]")
    B, H, D = q.shape
    G = k_cache.shape[1]
    if q.dtype not in _BF16 or not q.is_contiguous():
        _all(index, (("q", q, _BF16),))
    P, page, dt = _kv_caches(index, k_cache, v_cache, k_scale, v_scale, G, D)
    _indices(index, (("block_table", block_table), ("context_lens", context_lens)) if topk_idx is None else
             (("block_table", block_table), ("context_lens", context_lens), ("topk_idx", topk_idx)))
    if block_table.dim() != 2 or block_table.shape[0] != B or context_lens.shape != (B,):
        raise ValueError("block_table / context_lens shape mismatch")
    if topk_idx is not None and (topk_idx.dim() != 2 or topk_idx.shape[0] != B or topk_idx.shape[1] < 1):
        raise ValueError("topk_idx must be [B, K] with K >= 1")
    if _derivatives():
        _inference_only("kv_attention_decode", q, k_cache, v_cache, k_scale, v_scale)
    max_pages = block_table.shape[1]
    mcl = max_pages * page if max_context_len is None else int(max_context_len)
    if mcl >> 31:
        raise ValueError("max_context_len must be in [0, 2^31)")
    if _current_device() != index:
        with torch.cuda.device(index):
            return kv_attention_decode(q, k_cache, v_cache, block_table, context_lens, scale, topk_idx,
                                       max_context_len, k_scale, v_scale, want_lse, workspace)
    K = 0 if topk_idx is None else topk_idx.shape[1]
    out = torch.empty_like(q, dtype=torch.bfloat16)
    lse = q.new_empty((B, H), dtype=torch.float32) if want_lse else None
    nws = lib.indexer_kv_attention_decode_workspace_bytes(B, H, G, D, mcl, K, dt)
    ws = _scratch(workspace, nws, q)
    st = lib.indexer_kv_attention_decode(q.data_ptr(), BF16, k_cache.data_ptr(), _ptr(k_scale), v_cache.data_ptr(),
                                         _ptr(v_scale), dt, block_table.data_ptr(), max_pages, P,
                                         context_lens.data_ptr(), mcl, _ptr(topk_idx), K, B, H, G, D, page, scale,
                                         out.data_ptr(), _ptr(lse), _ptr(ws), nws, _raw_stream(index))
    if st:
        _lib.check(st, "indexer_kv_attention_decode")
    return out, lse
