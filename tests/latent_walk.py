"""Inputs on which the softmax's reference moves in the middle of a run of
tiles, and the walk over such a run in 64 bits, with mistakes that can be
planted in it.

A row of the pool has a level in column 0, by which every head's score rises: a
steep head of each 16 by some 20 bits a tile, past the slack of 2^16 that a
reference has, the others by at most three.  So the steep head moves the
references of its whole block at every tile, and the factors that the other
heads' sums then take are 1, 1/2, .. 1/8, which the results show."""
from __future__ import annotations

import numpy as np
import torch

from latent_util import V, bf16
from oracle.formats import fp8_e4m3_to_f64
from oracle.kcache import encode_e4m3

SLACK = 16.0
LN2 = np.log(2.0)


def levels(n, cycle):
    """Level of each of n keys: its tile's number in a cycle of tiles, rising within the tile."""
    j = np.arange(n)
    return (j // 64) % cycle + (j % 64) / 64.0


def make_rows(rng, level, E, kind, gain=0):
    """(stored rows, scales or None, fp64 rows) of these levels.  fp8 rows have
    scales of 2^0 .. 2^8 times the smallest that holds the row, all times 2^gain."""
    x = rng.normal(size=(len(level), E))
    x[:, 0] = level
    if kind == "bf16":
        t, v = bf16(x)
        return t, None, v
    scale = np.abs(x).max(1) / 448 * 2.0 ** rng.uniform(0, 8, size=len(level))
    scale = scale.astype(np.float32)
    codes = encode_e4m3(x / scale[:, None])
    scale = scale * np.float32(2.0 ** gain)
    return torch.from_numpy(codes), torch.from_numpy(scale), fp8_e4m3_to_f64(codes) * scale[:, None].astype(np.float64)


def make_q(rng, T, H, E, gain=0):
    """Queries (for a softmax scale of 1): slopes in column 0, little in the others."""
    bits = rng.uniform(-0.5, 3.0, size=(T, H))       # a tile, in base 2
    h = np.arange(H)
    bits[:, h % 16 == (5 * (h // 16) + 3) % 16] = rng.uniform(18.0, 22.0)
    if H < 4:
        bits[:, 0] = 20.0
    q = 0.02 * rng.normal(size=(T, H, E))
    q[:, :, 0] = bits * LN2
    return bf16(q * 2.0 ** -gain)


def round_bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).float().bfloat16().double().numpy()


def walk(q, rows, scales, scale, step, block=16, plant=None):
    """The kernels' walk over one run of keys in 64 bits but for P: steps of
    `step` keys, blocks of `block` rows whose references move together when a
    score of one passes its own by 2^SLACK, P rounded to bf16 (with a row's fp8
    scale in units of the first one's).  plant: "sums" or "outputs" keep what
    they summed before a move as it was, "both" do."""
    H = q.shape[0]
    s2 = scale * (q @ rows.T) / LN2
    by = np.ones(len(rows)) if scales is None else scales.astype(np.float64)
    shift = 0.0 if scales is None else np.log2(by[0])
    v = rows[:, :V] / by[:, None]
    out, lse = np.zeros((H, V)), np.zeros(H)
    for r in range(0, H, block):
        s = s2[r:r + block]
        m = np.full(len(s), -np.inf)
        l, o = np.zeros(len(s)), np.zeros((len(s), V))
        for j in range(0, len(rows), step):
            top = s[:, j:j + step].max(1)
            if (top > m + (SLACK - shift)).any():
                to = np.maximum(m, top + shift)
                f = np.where(np.isneginf(m), 0.0, np.exp2(m - to))
                m = to
                if plant not in ("sums", "both"):
                    l = l * f
                if plant not in ("outputs", "both"):
                    o = o * f[:, None]
            p = np.exp2(s[:, j:j + step] - m[:, None])
            l += p.sum(1)
            o += round_bf16(p * by[j:j + step]) @ v[j:j + step]
        out[r:r + block] = o / l[:, None]
        lse[r:r + block] = (m + np.log2(l)) * LN2
    return round_bf16(out), lse


def assert_tight(want, where):
    """The bounds that a test checks against are small next to what they bound:
    a tenth of each head's largest value, and of 1 for the lse."""
    for t, (o, _, eo, el) in enumerate(want):
        assert (eo.max(1) <= 0.1 * np.abs(o).max(1)).all() and (el <= 0.1).all(), f"{where}: loose bounds, query {t}"
