"""Infinities and NaN in the rows that kcache_append and cache_append_rope
quantise: an infinite element keeps its sign, a NaN in a latent row stays one,
and the other rows of the call are what they are without them."""
import numpy as np
import pytest
import torch

import dsa_lightning_indexer_03_amd as dsa
from gpu_util import say
from latent_util import bf16
from oracle.formats import fp8_e4m3_to_f64
from oracle.kcache import quantize_keys

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rows(rng, n, width, inp):
    """n rows whose elements behind column 64 are special in rows 0 .. 5, and what is special."""
    x = rng.normal(size=(n, width)).astype(np.float32)
    x[0, 70], x[1, 71] = INF, -INF
    x[2, 64:68] = INF, -INF, INF, -INF
    x[3, 80] = NAN
    x[4, 81], x[4, 90] = NAN, INF
    x[5] = 0
    x[5, 100] = 1e-44 if inp == "f32" else 9.2e-41   # a scale that underflows to 0, or a subnormal one
    return bf16(x)[1].astype(np.float32) if inp == "bf16" else x   # as the device has them


def device(x, inp):
    t = torch.from_numpy(x).cuda()
    return t.bfloat16() if inp == "bf16" else t


def place(n):
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    return torch.zeros(n, dtype=torch.int32, device="cuda"), pos, torch.zeros((1, 1), dtype=torch.int32, device="cuda")


def check(codes, scale, x, keep_nan):
    """Codes and scales of the rows x (without a rotation)."""
    got = fp8_e4m3_to_f64(codes)
    for i, row in enumerate(x):
        inf, nan = np.isinf(row), np.isnan(row)
        if inf.any():
            assert np.isposinf(scale[i]), f"row {i}"
            assert np.array_equal(codes[i][inf], np.where(row[inf] > 0, 0x7E, 0xFE)), f"row {i}: the infinities' codes"
            assert not got[i][~inf & ~nan].any(), f"row {i}: finite elements"
        else:
            with np.errstate(divide="ignore", invalid="ignore"):
                want, s = quantize_keys(np.where(nan, np.float32(0), row)[None])
            assert scale[i] == s[0], f"row {i}: scale {scale[i]} against {s[0]}"
            if s[0] > 0:
                assert np.array_equal(codes[i][~nan], want[0][~nan]), f"row {i}: codes"
            else:
                assert not codes[i][row == 0].any(), f"row {i}: zeros under a scale of 0"
        assert not np.isnan(got[i][~nan]).any()
        assert np.isnan(got[i][nan]).all() if keep_nan else not np.isnan(got[i]).any(), f"row {i}: NaN"


@pytest.mark.parametrize("inp", ["bf16", "f32"])
def test_kcache_append(inp):
    x = rows(np.random.default_rng(1), 40, 128, inp)
    say(f"kcache_append, infinities, {inp}")
    kc, ks = torch.zeros((1, 64, 128), dtype=torch.uint8, device="cuda"), torch.zeros((1, 64), device="cuda")
    dsa.kcache_append(device(x, inp), *place(40), kc, ks)
    torch.cuda.synchronize()
    check(kc.cpu().numpy()[0, :40], ks.cpu().numpy()[0], x, False)


@pytest.mark.parametrize("inp", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_cache_append_rope(inp, kind):
    """The special elements lie outside the 64 rotated columns of both rows; angle 0 leaves the others as they are."""
    rng = np.random.default_rng(2)
    E, n = 576, 40
    ix = rows(rng, n, 128, inp)
    kv = rng.normal(size=(n, E)).astype(np.float32)
    if inp == "bf16":
        kv = bf16(kv)[1].astype(np.float32)
    kv[:6, :512] = np.tile(rows(rng, n, 128, inp)[:6], (1, 4))
    kv[5, 512:] = 0
    cs = torch.cat([torch.ones(64, 32), torch.zeros(64, 32)], 1).cuda()
    say(f"cache_append_rope, infinities and NaN, {inp} to {kind}")
    latent = torch.zeros((1, 64, E), dtype=torch.bfloat16 if kind == "bf16" else torch.uint8, device="cuda")
    ls = torch.zeros((1, 64), device="cuda") if kind == "fp8" else None
    kc, ks = torch.zeros((1, 64, 128), dtype=torch.uint8, device="cuda"), torch.zeros((1, 64), device="cuda")
    seq, pos, table = place(n)
    dsa.cache_append_rope(device(kv, inp), seq, pos, table, latent, cs, latent_scale=ls, index_k=device(ix, inp),
                          k_cache=kc, k_scale=ks)
    torch.cuda.synchronize()
    check(kc.cpu().numpy()[0, :n], ks.cpu().numpy()[0], ix, False)
    if kind == "fp8":
        check(latent.cpu().numpy()[0, :n], ls.cpu().numpy()[0], kv, True)
    else:
        got = latent.cpu()[0, :n]
        assert torch.equal(got.view(torch.int16)[~torch.isnan(got)],
                           torch.from_numpy(kv).bfloat16().view(torch.int16)[~torch.isnan(got)])
        assert torch.equal(torch.isnan(got), torch.from_numpy(np.isnan(kv)))


def test_a_nan_reaches_the_attention():
    """The query that selects the row with a NaN among its values gives NaN there; its neighbour does not."""
    E, n = 576, 40
    g = torch.Generator(device="cuda").manual_seed(4)
    kv = torch.randn((n, E), generator=g, device="cuda")
    kv[7, 100] = NAN
    cs = torch.cat([torch.ones(64, 32), torch.zeros(64, 32)], 1).cuda()
    latent = torch.zeros((1, 64, E), dtype=torch.uint8, device="cuda")
    ls = torch.zeros((1, 64), device="cuda")
    seq, pos, table = place(n)
    dsa.cache_append_rope(kv, seq, pos, table, latent, cs, latent_scale=ls)
    q = torch.randn((2, 16, E), generator=g, device="cuda", dtype=torch.bfloat16)
    idx = torch.tensor([[7, 8], [8, 9]], dtype=torch.int32, device="cuda")
    out, _ = dsa.latent_attention_topk(q, latent, table, idx, 512, 0.04, latent_scale=ls, seq_ids=seq[:2].clone())
    torch.cuda.synchronize()
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isfinite(out[1]).all())
