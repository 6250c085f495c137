"""The operators around the selection, oracle side: the rotated write of the
two caches and attention over the paged latent cache, in fp64 (test
infrastructure; shares no code with the GPU path).

What the pages fix: the key path ends in a position rotation and an FP8
quantisation, the latent row carries its own rotated part, both caches are
written before the scoring decision (Study MLA Indexer, the data-flow diagram
and the notes on its two caches); the sparse attention reads the latent cache
at the selected positions only (the same diagram's last step; Lightning
Indexer explained, section 1).  The readings taken here:

* The last R columns of a latent row and the first R columns of an index key
  are rotated.  Pair i of the rotated part is columns (2i, 2i+1) or
  (i, i + R/2); (a, b) -> (a cos_i - b sin_i, b cos_i + a sin_i).
* All heads share the E-wide row; its first V columns are the value.
* A list of rows may name a row twice (it counts twice) or be empty (zeros,
  lse = -inf).  Page ids outside the pool, positions outside the table and
  sequence ids outside it name no row.

Each function also returns how far the fp32 computation with one rounding per
stored element (and bf16 probabilities) may be from the fp64 value, so that a
test's tolerance follows from the arithmetic: 2^-24 is half a step of fp32,
2^-8 of bf16, relative to the value.
"""
from __future__ import annotations

import numpy as np

U32, U16 = 2.0 ** -24, 2.0 ** -8


def rotate(x: np.ndarray, cos_sin: np.ndarray, first: int, pairs: bool):
    """x [T][n] fp64, cos_sin [T][R] -> (rotated [T][n], absolute bound of the
    fp32 result's error [T][n]).  An fp32 product pair and its sum are off by
    at most 2 half steps of |a| + |b| in the products (|cos|, |sin| <= 1) and
    one in the sum."""
    y = np.array(x, dtype=np.float64)
    err = np.zeros_like(y)
    R = cos_sin.shape[1]
    c, s = cos_sin[:, :R // 2].astype(np.float64), cos_sin[:, R // 2:].astype(np.float64)
    i = np.arange(R // 2)
    ia, ib = (first + 2 * i, first + 2 * i + 1) if pairs else (first + i, first + R // 2 + i)
    a, b = x[:, ia], x[:, ib]
    y[:, ia], y[:, ib] = a * c - b * s, b * c + a * s
    err[:, ia] = err[:, ib] = 3 * U32 * (np.abs(a) + np.abs(b))
    return y, err


def slots(seq_ids, positions, block_table, num_pages: int, limit: int | None = None, page_size: int = 64):
    """Slot of the pool for each (sequence, position), -1 where it names none."""
    out = np.full(len(seq_ids), -1, dtype=np.int64)
    top = block_table.shape[1] * page_size
    top = top if limit is None else min(top, limit)
    for i, (b, p) in enumerate(zip(seq_ids, positions)):
        if 0 <= b < block_table.shape[0] and 0 <= p < top:
            page = int(block_table[b, p // page_size])
            if 0 <= page < num_pages:
                out[i] = page * page_size + p % page_size
    return out


def attend(q: np.ndarray, rows: np.ndarray, scale: float, v_dim: int):
    """q [H][E], rows [n][E] fp64 -> (out [H][V], lse [H], bound of |out|'s
    error [H][V], bound of lse's error [H])."""
    H, n = q.shape[0], rows.shape[0]
    if n == 0:
        return np.zeros((H, v_dim)), np.full(H, -np.inf), np.zeros((H, v_dim)), np.zeros(H)
    s = scale * (q @ rows.T)
    m = s.max(axis=1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(axis=1, keepdims=True)
    p /= total
    v = rows[:, :v_dim]
    out = p @ v
    lse = (m + np.log(total))[:, 0]
    # a score: E products and sums, the row's scale, the softmax scale and the
    # subtraction of the maximum; then the exponential itself
    mag = abs(scale) * (np.abs(q) @ np.abs(rows).T).max(axis=1)
    ds = (q.shape[1] + 4) * U32 * mag + 8 * U32 * (np.abs(s).max(axis=1) + 1)
    rel = np.expm1(2 * ds) + U16 * (1 + np.expm1(2 * ds)) + (n + 16) * U32
    err = rel[:, None] * (p @ np.abs(v))
    err = err + U16 * (np.abs(out) + err)
    return out, lse, err, ds + (n + 16) * U32 + 4 * U32 * np.abs(lse)
