"""Inputs and checks shared by the tests of attention with grouped keys and values."""
from __future__ import annotations

import numpy as np
import torch

from oracle.formats import fp8_e4m3_to_f64
from oracle.kcache import encode_e4m3


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def bf16(x):
    """numpy -> torch bf16 tensor and its fp64 values."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16()
    return t, t.double().numpy()


def make_pool(rng, pages, G, D, kind, live=None):
    """(device cache, device scale or None, fp64 rows [pages][G][64][D]).  Slots
    (page, slot) not in `live` [pages][64] (None: all are) hold NaN, in fp8 pools
    the scale too."""
    x = rng.normal(size=(pages, G, 64, D))
    dead = np.zeros((pages, G, 64), bool) if live is None else np.broadcast_to(~live[:, None], (pages, G, 64)).copy()
    dead_t = torch.from_numpy(np.ascontiguousarray(dead))
    if kind == "bf16":
        t, v = bf16(x)
        t[dead_t] = float("nan")
        return t.cuda(), None, v
    codes = encode_e4m3(np.clip(x * 100, -448, 448))
    scale = rng.uniform(0.005, 0.015, size=(pages, G, 64)).astype(np.float32)
    v = fp8_e4m3_to_f64(codes) * scale[..., None].astype(np.float64)
    codes[dead] = 0x7F
    scale[dead] = np.nan
    return torch.from_numpy(codes).cuda(), torch.from_numpy(scale).cuda(), v


def check(out, lse, want, where):
    """Device results [rows][H][V], [rows][H] against a list of (out, lse, bounds of both)."""
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for t, (o, l, eo, el) in enumerate(want):
        d = np.abs(out[t] - o) - eo
        assert np.isfinite(out[t]).all() and (d <= 0).all(), f"{where}: out of row {t} off by {d.max():.3g} over its bound"
        none = np.isneginf(l)
        assert np.isneginf(lse[t][none]).all(), f"{where}: lse of the empty row {t}"
        assert (np.abs(lse[t][~none] - l[~none]) <= el[~none]).all(), f"{where}: lse of row {t}"
