"""kv_attention_decode's probabilities enter the product with the values in two
bf16 terms: outputs that cancel keep what one term would lose, and infinite values
come out as they are."""
import numpy as np
import pytest
import torch

import dsa_lightning_indexer_03_amd as dsa
from gpu_util import say
from kv_util import bf16, ints
from oracle.formats import fp8_e4m3_to_f64
from oracle.kcache import encode_e4m3

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def paged(x, table, pages):
    """[B][n][D] (n <= 64) -> pool [pages][1][64][D], each sequence's rows in its first page."""
    pool = np.full((pages, 1, 64, x.shape[2]), np.nan)
    for b, row in enumerate(table):
        pool[row[0], 0, :x.shape[1]] = x[b]
    return bf16(pool)[0].cuda()


@pytest.mark.parametrize("n", [2, 6, 40])
@pytest.mark.parametrize("R,B,mpp,listed", [(1, 2, 1, False), (1, 2, 1024, False), (8, 200, 1, False), (8, 2, 1, True),
                                            (24, 2, 1, False), (24, 3, 1024, False), (64, 2, 1, False),
                                            (64, 2, 1024, True)])
@pytest.mark.parametrize("D", [64, 128])
def test_values_that_cancel(D, R, B, mpp, listed, n):
    """Keys in pairs whose scores differ by a bf16 step, with values v and -v: the
    result is some 2^-9 of sum P |v|, so its own rounding, half a step of bf16 or
    2^-8 of it, is some 2^-17, where P in one bf16 term would be off by up to 2^-9.

    Bound: a probability's two terms.  The first keeps 7 bits behind the leading
    one, so the rest is less than 2^-7 of it, and is rounded by at most 2^-8 of
    itself: 2^-15.  A score is one product (the others are exact zeros) and its
    scaling, 2 roundings, and its maximum's subtraction, one more of a number below
    2^3 in base 2; with exp2's own error of at most 2 units that is 2 (3 * 2^-24 *
    2^3 + 2^-23) of the ratio of two probabilities, below 2^-18.  Sums of n products
    and their join are below (n + 16) * 2^-24."""
    rng = np.random.default_rng(n * R + D)
    qx = np.zeros((B, R, D))
    qx[:, :, 3] = rng.uniform(0.25, 1.0, size=(B, R))
    q, qv = bf16(qx)
    kx = np.zeros((B, n, D))
    near = rng.integers(128, 255, size=(B, n // 2)) / 128.0        # in [1, 2), and the next bf16 number
    kx[:, 0::2, 3], kx[:, 1::2, 3] = near, near + 1 / 128
    vx = bf16(rng.uniform(0.5, 2.0, size=(B, n // 2, D)))[1]
    vx = np.stack([vx, -vx], 2).reshape(B, n, D)
    pages = B + 1
    table = np.full((B, mpp), -1)
    table[:, 0] = rng.permutation(pages)[:B]
    order = np.stack([rng.permutation(n) for _ in range(B)])
    say(f"values that cancel: {n} keys, {R} heads, {D} columns, {B} x {mpp} pages, {'listed' if listed else 'all'}")
    out, lse = dsa.kv_attention_decode(q.cuda(), paged(kx, table, pages), paged(vx, table, pages), ints(table),
                                       ints([n] * B), 1.0, topk_idx=ints(order) if listed else None, want_lse=True)
    torch.cuda.synchronize()
    s = np.einsum("bhd,bnd->bhn", qv, kx)
    p = np.exp(s)
    p /= p.sum(2, keepdims=True)
    want, size = p @ vx, p @ np.abs(vx)
    err = (2.0 ** -15 + 2.0 ** -18 + (n + 16) * 2.0 ** -24) * size
    err += 2.0 ** -8 * (np.abs(want) + err)
    d = np.abs(out.double().cpu().numpy() - want)
    assert (d <= err).all(), f"off by {(d / err).max():.3g} of the bound"


@pytest.mark.parametrize("n", [1, 2, 37, 64])
@pytest.mark.parametrize("R", [1, 20, 64])
@pytest.mark.parametrize("mpp", [1, 1024])
def test_values_that_are_infinite(mpp, R, n):
    """An infinite value of a position that is seen makes its column infinite (of both
    signs, or NaN: NaN), whatever its probability's rest is, and changes no other."""
    rng = np.random.default_rng(n + R)
    D = 128
    q = bf16(rng.normal(size=(1, R, D)))[0].cuda()
    k, v = rng.normal(size=(1, n, D)), rng.normal(size=(1, n, D))
    table = np.full((1, mpp), -1)
    table[0, 0] = 1
    inf = v.copy()
    inf[0, 0, 5], inf[0, n // 2, 6], inf[0, n - 1, 7] = np.inf, -np.inf, np.nan
    inf[0, :, 8] = np.inf
    inf[0, n // 2, 9] = np.inf
    inf[0, 0, 9] = -np.inf if n > 1 else np.nan
    call = lambda v: dsa.kv_attention_decode(q, paged(k, table, 2), paged(v, table, 2), ints(table), ints([n]), 0.1,  # noqa: E731
                                             want_lse=True)
    say(f"infinite values: {n} keys, {R} heads, {mpp} pages")
    (want, l0), (out, l1) = call(v), call(inf)
    torch.cuda.synchronize()
    keep = [c for c in range(D) if c not in (5, 6, 7, 8, 9)]
    assert torch.equal(out[:, :, keep], want[:, :, keep]) and torch.equal(l0, l1)
    got = out[0].float().cpu().numpy()
    assert np.isposinf(got[:, [5, 8]]).all() and np.isneginf(got[:, 6]).all() and np.isnan(got[:, [7, 9]]).all()


@pytest.mark.parametrize("R", [1, 20, 64])
@pytest.mark.parametrize("mpp", [1, 1024])
def test_a_value_out_of_reach(mpp, R):
    """A position whose score is 300 below the others' has probability 0 in fp32, and
    takes no part, however large its value: e^-300 times bf16's largest is 1e-92."""
    rng = np.random.default_rng(R)
    n, D = 50, 128
    qx = np.zeros((1, R, D))
    qx[:, :, 0] = 1
    k, v = rng.normal(size=(1, n, D)), rng.normal(size=(1, n, D))
    k[0, :, 0], k[0, 20, 0] = 0, -300
    table = np.full((1, mpp), -1)
    table[0, 0] = 1
    q = bf16(qx)[0].cuda()
    call = lambda v: dsa.kv_attention_decode(q, paged(k, table, 2), paged(v, table, 2), ints(table), ints([n]), 1.0,  # noqa: E731
                                             want_lse=True)
    say(f"a value out of reach: {R} heads, {mpp} pages")
    v[0, 20] = 0
    want = call(v)
    v[0, 20] = np.where(np.arange(D) % 2, -1, 1) * 3.3e38
    out = call(v)
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def paged_codes(codes, scale, table, pages):
    """[B][n][D] codes, [B][n] scales -> pools, each sequence's rows in its first page; NaN elsewhere."""
    c, f = np.full((pages, 1, 64, codes.shape[2]), 0x7F, np.uint8), np.full((pages, 1, 64), np.nan, np.float32)
    for b, row in enumerate(table):
        c[row[0], 0, :codes.shape[1]], f[row[0], 0, :codes.shape[1]] = codes[b], scale[b]
    return torch.from_numpy(c).cuda(), torch.from_numpy(f).cuda()


@pytest.mark.parametrize("n", [2, 6, 40])
@pytest.mark.parametrize("R,B,mpp,listed", [(1, 2, 1, False), (1, 2, 1024, False), (8, 200, 1, False), (8, 2, 1, True),
                                            (24, 2, 1, False), (24, 3, 1024, False), (64, 2, 1, False),
                                            (64, 2, 1024, True)])
@pytest.mark.parametrize("D", [64, 128])
def test_fp8_values_that_cancel(D, R, B, mpp, listed, n):
    """As with bf16 rows: a key's one element is 1 and its scale the score's, the pair's
    values are one row and its negative under a scale of their own, of either sign and
    any size.

    Bound: as there, and three roundings for the scales (the key's product, the value's
    scale in the run's unit, its product with the probability) and one for the
    unit's reciprocal and the unit put back: 5 * 2^-24, below 2^-21."""
    rng = np.random.default_rng(n * R + D)
    qx = np.zeros((B, R, D))
    qx[:, :, 3] = rng.uniform(0.25, 1.0, size=(B, R))
    q, qv = bf16(qx)
    kc = np.zeros((B, n, D), np.uint8)
    kc[:, :, 3] = 0x38                                             # 1.0
    near = rng.integers(128, 255, size=(B, n // 2)) / 128.0
    ks = np.stack([near, near + 1 / 128], 2).reshape(B, n).astype(np.float32)
    vc = encode_e4m3(rng.uniform(100, 448, size=(B, n // 2, D)))
    vc = np.stack([vc, vc ^ 0x80], 2).reshape(B, n, D)
    vs = np.repeat(np.exp2(rng.uniform(-12, 12, size=(B, n // 2))), 2, axis=1).astype(np.float32)
    flip = rng.random((B, n)) < 0.3
    vs[flip] *= -1
    vc[flip] ^= 0x80
    pages = B + 1
    table = np.full((B, mpp), -1)
    table[:, 0] = rng.permutation(pages)[:B]
    order = np.stack([rng.permutation(n) for _ in range(B)])
    say(f"fp8 values that cancel: {n} keys, {R} heads, {D} columns, {B} x {mpp} pages, {'listed' if listed else 'all'}")
    (k, kf), (v, vf) = paged_codes(kc, ks, table, pages), paged_codes(vc, vs, table, pages)
    out, _ = dsa.kv_attention_decode(q.cuda(), k, v, ints(table), ints([n] * B), 1.0, k_scale=kf, v_scale=vf,
                                     topk_idx=ints(order) if listed else None, want_lse=True)
    torch.cuda.synchronize()
    p = np.exp(qv[:, :, 3:4] * ks.astype(np.float64)[:, None])
    p /= p.sum(2, keepdims=True)
    vx = fp8_e4m3_to_f64(vc) * vs.astype(np.float64)[..., None]
    want, size = p @ vx, p @ np.abs(vx)
    err = (2.0 ** -15 + 2.0 ** -18 + 2.0 ** -21 + (n + 16) * 2.0 ** -24) * size
    err += 2.0 ** -8 * (np.abs(want) + err)
    d = np.abs(out.double().cpu().numpy() - want)
    assert (d <= err).all(), f"off by {(d / err).max():.3g} of the bound"


@pytest.mark.parametrize("at", [0, 17])
@pytest.mark.parametrize("R", [1, 20, 64])
@pytest.mark.parametrize("mpp", [1, 1024])
def test_an_infinite_scale(mpp, R, at):
    """A value row that was written with infinite elements has an infinite scale: these
    read as themselves, the others, codes of 0, as NaN."""
    rng = np.random.default_rng(R)
    n, D = 33, 128
    q = bf16(rng.normal(size=(1, R, D)))[0].cuda()
    kc, vc = (encode_e4m3(rng.uniform(-448, 448, size=(1, n, D))) for _ in range(2))
    ks, vs = (rng.uniform(0.002, 0.004, size=(1, n)).astype(np.float32) for _ in range(2))
    vc[0, at] = 0
    vc[0, at, 7], vc[0, at, 90] = 0x7E, 0xFE                       # 448 and -448
    vs[0, at] = np.inf
    table = np.full((1, mpp), -1)
    table[0, 0] = 1
    say(f"an infinite scale: {R} heads, {mpp} pages, row {at}")
    (k, kf), (v, vf) = paged_codes(kc, ks, table, 2), paged_codes(vc, vs, table, 2)
    out, lse = dsa.kv_attention_decode(q, k, v, ints(table), ints([n]), 0.1, k_scale=kf, v_scale=vf, want_lse=True)
    torch.cuda.synchronize()
    got = out[0].float().cpu().numpy()
    assert bool(lse.isfinite().all()) and np.isposinf(got[:, 7]).all() and np.isneginf(got[:, 90]).all()
    assert np.isnan(np.delete(got, [7, 90], axis=1)).all()
