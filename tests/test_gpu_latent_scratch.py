"""A workspace's contents on entry do not matter: calls in several parts, some
of which no key reaches, on a workspace of NaN, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import dsa_lightning_indexer_03_amd as dsa
from gpu_util import say
from latent_util import V, bf16, check_attention, expect_topk, make_pool
from oracle.latent import attend

pytestmark = pytest.mark.gpu
E, SCALE = 576, 576 ** -0.5


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def poisoned(nbytes, rows):
    """A workspace of NaN with room behind it, and the parts that it holds."""
    parts = nbytes // (rows * 514 * 4)
    assert parts > 1, f"{parts} parts"
    return torch.full((nbytes + 64,), 0xFF, dtype=torch.uint8, device="cuda"), parts


# rows of T * H below 2048, where four waves join a row, and from there on, where one does
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("T,H", [(9, 16), (7, 32), (5, 64), (6, 100), (128, 16), (65, 32), (33, 64), (20, 110)])
def test_selections_with_parts_of_nothing(T, H, kind):
    rng = np.random.default_rng(T * H)
    mpp, K = 4, 2300
    pages = T * mpp
    table = rng.permutation(pages).reshape(T, mpp)
    idx = rng.integers(0, mpp * 64, (T, K))
    idx[0] = -1                          # a query without a row: no part holds anything
    idx[1, 64:] = -1                     # the first part alone
    idx[2, :-20] = -1                    # the last alone
    idx[3, 100:-100] = -1                # none in between
    idx[4, :-1] = -1                     # one row, in the last
    cache, scale, rows = make_pool(rng, pages, E, kind)
    q, qv = bf16(1.5 * rng.normal(size=(T, H, E)))
    nbytes = dsa.latent_topk_workspace_bytes(T, H, E, V, K, kind == "fp8")
    ws, parts = poisoned(nbytes, T * H)
    say(f"{T} queries of {H} heads, {parts} parts on a workspace of NaN, {kind}")
    out, lse = dsa.latent_attention_topk(q.cuda(), cache, ints(table), ints(idx), V, SCALE, latent_scale=scale,
                                         want_lse=True, workspace=ws)
    torch.cuda.synchronize()
    assert bool((ws[nbytes:] == 0xFF).all())
    check_attention(out, lse, expect_topk(qv, rows, table, idx, np.arange(T), SCALE, pages), f"T={T} H={H} {kind}")


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("B,H", [(6, 16), (70, 5), (5, 64), (300, 8), (40, 64), (18, 128)])
def test_prefix_and_own_parts_of_nothing(B, H, kind):
    """Own keys of no sequence, of some and of every length, bad pages of the prefix, on a workspace of NaN."""
    rng = np.random.default_rng(B * H)
    mpp, prefix = 6, 64 * 30 - 11
    n_pre = 30
    pages = n_pre + 40
    ptab = rng.permutation(n_pre)
    table = n_pre + rng.integers(0, 40, (B, mpp))
    lens = rng.integers(0, mpp * 64 + 1, B)
    lens[0], lens[1], lens[2] = 0, 64 * mpp, 1
    ptab[4:12] = -1                      # parts of the prefix without a row
    cache, scale, rows = make_pool(rng, pages, E, kind)
    q, qv = bf16(1.5 * rng.normal(size=(B, H, E)))
    nbytes = dsa.latent_shared_workspace_bytes(B, H, E, V, prefix, mpp * 64, kind == "fp8")
    ws, parts = poisoned(nbytes, B * H)
    say(f"{B} queries of {H} heads, {parts} parts on a workspace of NaN, {kind}")
    out, lse = dsa.latent_attention_shared(q.cuda(), cache, ints(ptab), prefix, ints(table), ints(lens), V, SCALE,
                                           latent_scale=scale, want_lse=True, workspace=ws)
    torch.cuda.synchronize()
    assert bool((ws[nbytes:] == 0xFF).all())
    s = np.arange(prefix)
    pre = ptab[s // 64] * 64 + s % 64
    pre = pre[ptab[s // 64] >= 0]
    want = []
    for b in range(B):
        s = np.arange(lens[b])
        want.append(attend(qv[b], rows[np.concatenate([pre, table[b, s // 64] * 64 + s % 64])], SCALE, V))
    check_attention(out, lse, want, f"B={B} H={H} {kind}")


@pytest.mark.parametrize("H", [16, 64, 128])
def test_nothing_at_all(H):
    """No query has a key, and every part is empty: zeros and -inf."""
    T, K, prefix = 4, 900, 64 * 20
    g = torch.Generator(device="cuda").manual_seed(H)
    q = torch.randn((T, H, E), generator=g, device="cuda").bfloat16()
    cache = torch.full((3, 64, E), float("nan"), dtype=torch.bfloat16, device="cuda")
    table = ints(np.full((T, 8), -1))
    say(f"no key for any of {H} heads")
    ws, _ = poisoned(dsa.latent_topk_workspace_bytes(T, H, E, V, K), T * H)
    idx = ints(np.tile(np.arange(K) % 512, (T, 1)))
    got = dsa.latent_attention_topk(q, cache, table, idx, V, SCALE, want_lse=True, workspace=ws)
    ws, _ = poisoned(dsa.latent_shared_workspace_bytes(T, H, E, V, prefix, 512), T * H)
    got += dsa.latent_attention_shared(q, cache, ints(np.full(20, 3)), prefix, table, ints([0, 512, 5, 64]), V, SCALE,
                                       want_lse=True, workspace=ws)
    torch.cuda.synchronize()
    for out, lse in (got[:2], got[2:]):
        assert not bool(out.any()) and bool(torch.isneginf(lse).all())
