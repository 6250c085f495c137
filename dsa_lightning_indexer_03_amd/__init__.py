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

Input formats: fp32 tensors; bf16 as torch.bfloat16 or int16/uint16 bit
patterns; OCP FP8 E4M3 as torch.float8_e4m3fn or uint8 codes with fp32
per-row scales.
"""
from __future__ import annotations

import torch

from . import _lib

F32, BF16, FP8_E4M3 = 0, 1, 2

__all__ = ["indexer_prefill", "indexer_prefill_noalloc", "indexer_decode_paged", "topk_select", "kcache_append", "topk_gather",
           "topk_gather_layers",
           "prefill_chunk_paged", "prefill_chunk_varlen",
           "cache_append_rope", "latent_attention_topk", "latent_attention_shared", "latent_topk_workspace_bytes",
           "latent_shared_workspace_bytes", "dtype_code", "F32", "BF16", "FP8_E4M3"]


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


def _inference_only(where: str, *tensors) -> None:
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{where} has no backward: call it under torch.no_grad() or detach its inputs")


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
