"""Attention with keys and values of their own for groups of heads, oracle
side: the rotated write of the two caches, causal attention over packed prompts
and one new token per sequence over the paged caches, in fp64 (test
infrastructure; shares no code with the GPU path).

Readings taken here (the pages write main attention as ordinary multi-head
attention and name its grouped form only in comparisons):

* Query head h reads key/value head h // (H / G).
* Row i of a packed sequence sees its rows 0 .. i (the lower-triangular mask of
  "From principle to code", section 3); rows behind the last sequence see none.
* No row: zeros, lse = -inf.  A list may name a position twice (it counts twice).
* The first R columns of a key are rotated, pair i being columns (2i, 2i+1) or
  (i, i + R/2); values are not.

Each function also returns how far the fp32 computation with one rounding per
stored element (and bf16 probabilities) may be from the fp64 value: 2^-24 is
half a step of fp32, 2^-8 of bf16, relative to the value.
"""
from __future__ import annotations

import numpy as np

U32, U16 = 2.0 ** -24, 2.0 ** -8


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float):
    """q [R][D] over keys k [n][D] and values v [n][V], fp64 -> (out [R][V],
    lse [R], bound of |out|'s error [R][V], bound of lse's error [R])."""
    R, n = q.shape[0], k.shape[0]
    if n == 0:
        return np.zeros((R, v.shape[1])), np.full(R, -np.inf), np.zeros((R, v.shape[1])), np.zeros(R)
    s = scale * (q @ k.T)
    m = s.max(axis=1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(axis=1, keepdims=True)
    p /= total
    out = p @ v
    lse = (m + np.log(total))[:, 0]
    # a score: D products and sums, the row's scale, the softmax's scale; the
    # subtraction of the reference and the exponential itself
    mag = abs(scale) * (np.abs(q) @ np.abs(k).T).max(axis=1)
    ds = (q.shape[1] + 4) * U32 * mag + 8 * U32 * (np.abs(s).max(axis=1) + 1)
    rel = np.expm1(2 * ds) + U16 * (1 + np.expm1(2 * ds)) + (n + 16) * U32
    err = rel[:, None] * (p @ np.abs(v))
    err = err + U16 * (np.abs(out) + err)
    return out, lse, err, ds + (n + 16) * U32 + 4 * U32 * np.abs(lse)


def grouped(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float):
    """One query's heads q [H][D] over keys k [n][G][D], values v [n][G][V]."""
    G = k.shape[1]
    R = q.shape[0] // G
    parts = [attend(q[g * R:(g + 1) * R], k[:, g], v[:, g], scale) for g in range(G)]
    return tuple(np.concatenate([p[i] for p in parts]) for i in range(4))


def prompt(q: np.ndarray, k: np.ndarray, v: np.ndarray, cu, scale: float):
    """q [T][H][D], k [T][G][D], v [T][G][V], cu [B+1] -> grouped()'s four arrays for every row."""
    T, H = q.shape[:2]
    V = v.shape[2]
    out, lse = np.zeros((T, H, V)), np.full((T, H), -np.inf)
    eo, el = np.zeros((T, H, V)), np.zeros((T, H))
    for a, b in zip(cu, cu[1:]):
        for i in range(a, b):
            out[i], lse[i], eo[i], el[i] = grouped(q[i], k[a:i + 1], v[a:i + 1], scale)
    return out, lse, eo, el


def positions(idx, ctx: int):
    """The positions that a list names: those inside the context, in order."""
    idx = np.asarray(idx, dtype=np.int64)
    return idx[(idx >= 0) & (idx < ctx)]


def place(pos, row, num_pages: int, page_size: int = 64):
    """(page, slot) of positions `pos` of a sequence with table row `row`; page -1: none."""
    pos = np.asarray(pos, dtype=np.int64)
    page = np.asarray(row, dtype=np.int64)[pos // page_size]
    return np.where((page >= 0) & (page < num_pages), page, -1), pos % page_size


def decode(q: np.ndarray, k: np.ndarray, v: np.ndarray, table, lens, scale: float, idx=None):
    """q [B][H][D], pools k, v [P][G][page][D] fp64 -> a list of grouped()'s results."""
    got = []
    for b in range(q.shape[0]):
        pos = np.arange(lens[b]) if idx is None else positions(idx[b], lens[b])
        page, slot = place(pos, table[b], k.shape[0], k.shape[2])
        page, slot = page[page >= 0], slot[page >= 0]
        got.append(grouped(q[b], k[page, :, slot], v[page, :, slot], scale))
    return got
