"""Attention over the latent cache with softmaxes that one row holds, or a few
of the same score, at inputs whose scores are exact: every value within the two
roundings to bf16 and little more."""
import numpy as np
import pytest
import torch

import dsa_lightning_indexer_03_amd as dsa
from gpu_util import say
from latent_util import V, bf16
from oracle.formats import fp8_e4m3_to_f64
from oracle.kcache import encode_e4m3

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def pool(t, scale, E):
    n = -len(t) % 64
    t = torch.cat([t, t[:n]]).view(-1, 64, E).cuda()
    return t, None if scale is None else torch.cat([scale, scale[:n]]).view(-1, 64).cuda()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("scale", [30.0, -7.0])
@pytest.mark.parametrize("T,H", [(3, 5), (300, 16), (2, 32), (260, 24), (3, 64), (257, 64), (2, 128), (256, 100)])
def test_one_row_holds_the_weight(T, H, scale, kind):
    """Rows and queries of small whole numbers (fp8: times powers of two), so
    that scores are exact in fp32, and distinct scores are at least 7 apart after
    the scale: the softmax is the mean over the rows of the highest score, plus
    less than 700 e^-7 of anything else, which the fp64 softmax counts.

    Tolerance, relative to the values that are averaged: P is rounded to bf16
    (2^-8), the output too (2^-8).  An exponent, |scale| log2(e) score - m, has
    one rounding of the factor, one of m and one of the difference: scores here
    stay below 64, so exponents below 64 * 30 * 1.45 < 2^12, each off by 2^-12
    at most, together 3 * 2^-12 in base 2, ln 2 of that in the value, for P and
    for its sum: 2^-9 holds both (2 * 3 * 2^-12 * 0.7 = 1.03 * 2^-10).  Weights
    below 2^-126 may be lost as fp32's subnormals: 700 of them on values of 16
    at most, 700 * 16 * 2^-126 < 2^-112, are all that some columns hold.  The lse
    is off by the roundings of the factor and m, 2 * 2^-24 of it, the sum's 2^-9
    in its logarithm, and its own few roundings: 2^-22 of it and 2^-9."""
    rng = np.random.default_rng(T + H)
    E, n = 576, 700
    x = np.zeros((n, E))
    x[:, :V] = rng.integers(-8, 9, size=(n, V))
    qx = np.zeros((T, H, E))
    for t in range(T):
        for h in range(H):   # three columns of ones: |score| <= 24
            qx[t, h, rng.choice(V, 3, replace=False)] = rng.choice([-1.0, 1.0], 3)
    if kind == "bf16":
        cache, rows = bf16(x)
        cs = None
    else:
        codes = encode_e4m3(x)
        s = 2.0 ** rng.integers(0, 2, size=n)   # scores of rows scaled by 2 stay below 64
        rows = fp8_e4m3_to_f64(codes) * s[:, None]
        cache, cs = torch.from_numpy(codes), torch.from_numpy(s.astype(np.float32))
    cache, cs = pool(cache, cs, E)
    q, qv = bf16(qx)
    idx = np.stack([rng.permutation(n) for _ in range(T)])
    say(f"one row holds the weight, T={T} H={H} scale={scale} {kind}")
    out, lse = dsa.latent_attention_topk(q.cuda(), cache, ints(np.arange(11)[None]), ints(idx), V, scale,
                                         latent_scale=cs, seq_ids=ints(np.zeros(T)), want_lse=True)
    torch.cuda.synchronize()
    for t in sorted({0, 1, T // 2, T - 1}):
        s = scale * (qv[t] @ rows.T)
        assert np.abs(s).max() < 64 * 30
        p = np.exp(s - s.max(1, keepdims=True))
        total = p.sum(1, keepdims=True)
        p /= total
        want, mag = p @ rows[:, :V], p @ np.abs(rows[:, :V])
        d = np.abs(out[t].double().cpu().numpy() - want)
        assert (d <= mag * (2 * 2.0 ** -8 + 2.0 ** -9) + 2.0 ** -112).all(), f"query {t}: {(d / np.maximum(mag, 1e-9)).max():.3g}"
        wl = s.max(1) + np.log(total[:, 0])
        assert (np.abs(lse[t].double().cpu().numpy() - wl) <= 2.0 ** -22 * np.abs(wl) + 2.0 ** -9).all(), f"lse of {t}"
