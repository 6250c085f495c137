"""The largest calls that the header lists: 2^23 rows of T * H, selections of
131072 entries, tables far wider than the contexts, 2^25 new tokens.  The
last rows are compared with the oracle, or with a small call on the same data."""
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


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("T,H", [(1 << 23, 1), (1 << 18, 32), (1 << 16, 128)])
def test_as_many_rows_as_a_call_takes(T, H, kind):
    """9.7 GB of queries, 8.6 GB of results: every query the same as one of 97."""
    rng = np.random.default_rng(H)
    pages, K = 4, 5
    cache, cs, _ = make_pool(rng, pages, E, kind)
    few = bf16(rng.normal(size=(97, H, E)))[0].cuda()
    some = ints(rng.integers(-1, 128, (97, K)))
    table = ints([[0, 1], [2, 3]])
    seq = ints(np.arange(97) % 2)
    say(f"{T} queries of {H} heads, {kind}")
    want, wl = dsa.latent_attention_topk(few, cache, table, some, V, SCALE, latent_scale=cs, seq_ids=seq, want_lse=True)
    at = torch.arange(T, device="cuda") % 97
    out, lse = dsa.latent_attention_topk(few[at], cache, table, some[at], V, SCALE, latent_scale=cs, seq_ids=seq[at],
                                         want_lse=True)
    torch.cuda.synchronize()
    assert bool(want.any()) and torch.equal(lse, wl[at])
    for i in range(0, T, T // 16):   # (a comparison of all at once would take another 25 GB)
        assert torch.equal(out[i:i + T // 16], want[at[i:i + T // 16]]), f"queries from {i}"


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("H", [2, 30, 60, 128])
def test_the_longest_selection(H, kind):
    rng = np.random.default_rng(H)
    mpp, K = 2100, 131072
    cache, cs, rows = make_pool(rng, mpp, E, kind)
    table = rng.permutation(mpp)[None]
    idx = rng.permutation(mpp * 64)[None, :K]
    q, qv = bf16(1.5 * rng.normal(size=(1, H, E)))
    say(f"{K} selected positions, {H} heads, {kind}")
    out, lse = dsa.latent_attention_topk(q.cuda(), cache, ints(table), ints(idx), V, SCALE, latent_scale=cs, want_lse=True)
    torch.cuda.synchronize()
    check_attention(out, lse, expect_topk(qv, rows, table, idx, [0], SCALE, mpp), f"H={H} {kind}")


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("B,H,prefix", [(3, 16, 0), (3, 16, 700), (9, 40, 1000), (2, 128, 64), (40, 16, 5000)])
def test_tables_far_wider_than_the_contexts(B, H, prefix, kind):
    """A table of 2^21 entries a sequence, the widest, and no max_context_len: ids
    behind the contexts name no page, and none of them is read."""
    rng = np.random.default_rng(B + prefix)
    n_pre = -(-prefix // 64)
    lens = rng.integers(0, 300, B)
    pages = n_pre + 5 * B
    cache, cs, rows = make_pool(rng, pages, E, kind)
    own = n_pre + rng.permutation(5 * B).reshape(B, 5)
    table = torch.full((B, 1 << 21), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    table[:, :5] = ints(own)
    ptab = np.arange(n_pre)
    q, qv = bf16(1.5 * rng.normal(size=(B, H, E)))
    say(f"tables of 2^21 pages, B={B} H={H} prefix={prefix} {kind}")
    out, lse = dsa.latent_attention_shared(q.cuda(), cache, ints(ptab) if n_pre else None, prefix, table, ints(lens), V,
                                           SCALE, latent_scale=cs, want_lse=True)
    torch.cuda.synchronize()
    want = []
    for b in range(B):
        s = np.arange(lens[b])
        want.append(attend(qv[b], rows[np.concatenate([np.arange(prefix), own[b, s // 64] * 64 + s % 64])], SCALE, V))
    check_attention(out, lse, want, f"B={B} H={H} prefix={prefix} {kind}")


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_as_many_tokens_as_a_call_takes(kind):
    """2^25 rows of 16 columns; all but the first and the last 64 are padding."""
    T, width = 1 << 25, 16
    g = torch.Generator(device="cuda").manual_seed(9)
    kv = torch.zeros((T, width), dtype=torch.bfloat16, device="cuda")
    kv[:64] = torch.randn((64, width), generator=g, device="cuda").bfloat16()
    kv[-64:] = torch.randn((64, width), generator=g, device="cuda").bfloat16()
    seq = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    here = torch.arange(64, dtype=torch.int32, device="cuda")
    seq[:64], seq[-64:], pos[:64], pos[-64:] = 0, 0, here, 64 + here
    ang = torch.rand((128, width // 2), generator=g, device="cuda")
    cs = torch.cat([ang.cos(), ang.sin()], 1)
    table = ints([[2, 1]])
    say(f"{T} tokens, {kind}")
    got = []
    few = torch.cat([torch.arange(64, device="cuda"), torch.arange(T - 64, T, device="cuda")])
    for part in (slice(None), few):
        latent = torch.full((3, 64, width), 1, dtype=torch.bfloat16 if kind == "bf16" else torch.uint8, device="cuda")
        ls = torch.full((3, 64), 7.0, device="cuda") if kind == "fp8" else None
        dsa.cache_append_rope(kv[part], seq[part], pos[part], table, latent, cs, latent_scale=ls)
        got.append((latent, ls))
    torch.cuda.synchronize()
    (a, sa), (b, sb) = got
    assert torch.equal(a, b) and bool((a[0] == 1).all()) and not bool((a[1:] == 1).all(-1).any())
    assert kind == "bf16" or torch.equal(sa, sb)
