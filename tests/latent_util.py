"""Inputs and checks shared by the tests of the operators on the latent cache."""
from __future__ import annotations

import numpy as np
import torch

from oracle.formats import fp8_e4m3_to_f64
from oracle.kcache import encode_e4m3
from oracle.latent import attend, slots

V = 512


def bf16(x):
    """numpy -> torch bf16 tensor and its fp64 values."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16()
    return t, t.double().numpy()


def make_pool(rng, pages, E, kind, used=None):
    """(device cache, device scale or None, fp64 rows [pages*64][E]).  Slots not
    in `used` (None: all are) hold NaN, in fp8 pools the scale too."""
    x = rng.normal(size=(pages * 64, E))
    dead = np.zeros(pages * 64, bool)
    if used is not None:
        dead[:] = True
        dead[np.asarray(used, dtype=np.int64)] = False
    if kind == "bf16":
        t, v = bf16(x)
        t[torch.from_numpy(dead)] = float("nan")
        return t.view(pages, 64, E).cuda(), None, v
    codes = encode_e4m3(np.clip(x * 100, -448, 448))
    scale = rng.uniform(0.005, 0.015, size=pages * 64).astype(np.float32)
    v = fp8_e4m3_to_f64(codes) * scale[:, None].astype(np.float64)
    codes[dead] = 0x7F
    scale[dead] = np.nan
    return (torch.from_numpy(codes).view(pages, 64, E).cuda(), torch.from_numpy(scale).view(pages, 64).cuda(), v)


def expect_topk(q, rows, table, idx, seq, scale, pages):
    """fp64 results of every query: lists of (out, lse, tol_out, tol_lse)."""
    got = []
    for t in range(q.shape[0]):
        s = slots(np.full(idx.shape[1], seq[t]), idx[t], table, pages)
        got.append(attend(q[t], rows[s[s >= 0]], scale, V))
    return got


def check_attention(out, lse, want, where):
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for t, (o, l, eo, el) in enumerate(want):
        d = np.abs(out[t] - o) - eo
        assert np.isfinite(out[t]).all() and (d <= 0).all(), f"{where}: out of query {t} off by {d.max():.3g} over its bound"
        if np.isneginf(l).any():
            assert np.isneginf(lse[t]).all(), f"{where}: lse of the empty query {t}"
        else:
            assert (np.abs(lse[t] - l) <= el).all(), f"{where}: lse of query {t}: {np.abs(lse[t] - l).max():.3g} > {el.min():.3g}"
