"""GPU parity of latent_attention_topk and latent_attention_shared against the
fp64 oracle, each value within the bound that the oracle derives from the
arithmetic.  Slots of the pool that no query may read hold NaN."""
import numpy as np
import pytest
import torch

import dsa_lightning_indexer_03_amd as dsa
from gpu_util import say
from latent_util import V, bf16, check_attention, expect_topk, make_pool
from oracle.latent import attend, slots

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make_topk(rng, T, H, K, E, kind, B=3, mpp=9, holes=0.0, q_scale=1.5):
    pages = B * mpp + 2
    table = rng.permutation(pages)[: B * mpp].reshape(B, mpp).astype(np.int32)
    idx = rng.integers(0, mpp * 64, size=(T, K)).astype(np.int32)
    idx[rng.random((T, K)) < holes] = -1
    seq = rng.integers(0, B, T).astype(np.int32)
    return dict(table=table, idx=idx, seq=seq, pages=pages, q=bf16(q_scale * rng.normal(size=(T, H, E))))


def run_topk(rng, d, E, kind, scale, where):
    used = np.unique(np.concatenate([slots(np.full(d["idx"].shape[1], s), i, d["table"], d["pages"])
                                     for s, i in zip(d["seq"], d["idx"])]))
    cache, cs, rows = make_pool(rng, d["pages"], E, kind, used[used >= 0])
    out, lse = dsa.latent_attention_topk(d["q"][0].cuda(), cache, torch.from_numpy(d["table"]).cuda(),
                                         torch.from_numpy(d["idx"]).cuda(), V, scale, latent_scale=cs,
                                         seq_ids=torch.from_numpy(d["seq"]).cuda(), want_lse=True)
    torch.cuda.synchronize()
    want = expect_topk(d["q"][1], rows, d["table"], d["idx"], d["seq"], scale, d["pages"])
    check_attention(out, lse, want, where)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("T,H,K,E", [
    (1, 1, 1, 576), (1, 16, 64, 576), (2, 17, 65, 512), (3, 5, 63, 576), (4, 33, 300, 512), (2, 64, 129, 576),
    (3, 128, 500, 576), (1, 100, 2048, 512), (70, 16, 40, 576), (5, 65, 1000, 576), (300, 48, 70, 512)])
def test_topk_random(T, H, K, E, kind):
    rng = np.random.default_rng(T * 7 + H * 13 + K)
    say(f"topk attention T={T} H={H} K={K} E={E} {kind}")
    run_topk(rng, make_topk(rng, T, H, K, E, kind), E, kind, E ** -0.5, f"T={T} H={H} K={K}")


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("H", [3, 32, 128])
def test_topk_holes_and_empty_rows(H, kind):
    """-1 anywhere in a row, rows without any entry, tiles without any entry,
    positions past the table, pages outside the pool, queries without a sequence."""
    rng = np.random.default_rng(H)
    d = make_topk(rng, 12, H, 400, 576, kind, holes=0.5)
    d["idx"][0] = -1                        # nothing selected
    d["idx"][1, 64:] = -1                   # only the first tile
    d["idx"][2, :330] = -1                  # only the last
    d["idx"][3] = -1
    d["idx"][3, 399] = 7                    # one entry, at the very end
    d["idx"][4, ::2] = 9 * 64 + d["idx"][4, ::2]   # past the table
    d["idx"][5, 0] = 2 ** 31 - 1
    d["idx"][5, 1] = -2 ** 31
    d["idx"][6] = 5                         # one position 400 times
    d["seq"][7], d["seq"][8] = -1, 3
    d["table"][0, :] = -1                   # a sequence without pages
    d["table"][1, 4] = d["pages"]
    d["seq"][9] = 0
    d["idx"][10, 100:] = -1
    say(f"topk attention with holes H={H} {kind}")
    run_topk(rng, d, 576, kind, 0.05, f"holes H={H}")


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.04, 30.0])
def test_topk_softmax_extremes(scale):
    """Uniform, peaked (one row holds all the weight) and reversed softmaxes,
    and scores that rise so that the running maximum changes at every tile."""
    rng = np.random.default_rng(11)
    d = make_topk(rng, 4, 20, 512, 576, "bf16", q_scale=1.0)
    say(f"topk attention scale={scale}")
    run_topk(rng, d, 576, "bf16", scale, f"scale={scale}")


def test_topk_rising_and_falling_scores():
    E, H, K = 576, 16, 576
    rng = np.random.default_rng(12)
    x = 0.05 * rng.normal(size=(9 * 64, E))
    x[:, 0] = np.linspace(-40, 40, 9 * 64)
    t, rows = bf16(x)
    q = 0.1 * rng.normal(size=(2, H, E))
    q[0, :, 0], q[1, :, 0] = 3.0, -3.0
    qt, qv = bf16(q)
    table = np.arange(9, dtype=np.int32)[None]
    idx = np.tile(np.arange(K, dtype=np.int32), (2, 1))
    out, lse = dsa.latent_attention_topk(qt.cuda(), t.view(9, 64, E).cuda(), torch.from_numpy(table).cuda(),
                                         torch.from_numpy(idx).cuda(), V, 1.0,
                                         seq_ids=torch.zeros(2, dtype=torch.int32, device="cuda"), want_lse=True)
    torch.cuda.synchronize()
    check_attention(out, lse, expect_topk(qv, rows, table, idx, [0, 0], 1.0, 9), "rising and falling")


def test_topk_without_seq_ids_and_lse():
    rng = np.random.default_rng(13)
    d = make_topk(rng, 3, 16, 100, 576, "bf16")
    d["seq"] = np.arange(3, dtype=np.int32)
    cache, _, rows = make_pool(rng, d["pages"], 576, "bf16")
    args = (d["q"][0].cuda(), cache, torch.from_numpy(d["table"]).cuda(), torch.from_numpy(d["idx"]).cuda(), V, 0.04)
    out, none = dsa.latent_attention_topk(*args)
    with_lse, lse = dsa.latent_attention_topk(*args, want_lse=True)
    torch.cuda.synchronize()
    assert none is None and torch.equal(out, with_lse)
    check_attention(out, lse, expect_topk(d["q"][1], rows, d["table"], d["idx"], d["seq"], 0.04, d["pages"]), "no seq_ids")


def run_shared(rng, B, H, E, kind, prefix, lens, scale, mpp=None, max_ctx=None, bad_pages=False, q_scale=1.5):
    lens = np.asarray(lens, dtype=np.int32)
    n_pre = -(-prefix // 64)
    mpp = mpp or max(1, -(-int(lens.max(initial=0)) // 64))
    pages = n_pre + B * mpp + 1
    perm = rng.permutation(pages).astype(np.int32)
    ptab, table = perm[:n_pre], perm[n_pre:n_pre + B * mpp].reshape(B, mpp)
    if bad_pages:
        ptab[0], table[0, 0] = -1, pages
    top = mpp * 64 if max_ctx is None else max_ctx
    pre = slots(np.zeros(prefix, int), np.arange(prefix), ptab[None] if n_pre else np.zeros((1, 1), np.int32), pages)
    own = [slots(np.full(n, b), np.arange(n), table, pages) for b, n in enumerate(np.clip(lens, 0, top))]
    used = np.concatenate([pre] + own)
    cache, cs, rows = make_pool(rng, pages, E, kind, used[used >= 0])
    q, qv = bf16(q_scale * rng.normal(size=(B, H, E)))
    out, lse = dsa.latent_attention_shared(q.cuda(), cache, torch.from_numpy(ptab).cuda() if n_pre else None, prefix,
                                           torch.from_numpy(np.ascontiguousarray(table)).cuda(),
                                           torch.from_numpy(lens).cuda(), V, scale, max_context_len=max_ctx,
                                           latent_scale=cs, want_lse=True)
    torch.cuda.synchronize()
    want = []
    for b in range(B):
        s = np.concatenate([pre, own[b]])
        want.append(attend(qv[b], rows[s[s >= 0]], scale, V))
    check_attention(out, lse, want, f"shared B={B} H={H} prefix={prefix}")


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("B,H,E,prefix,lens", [
    (1, 1, 576, 0, [0]), (1, 1, 576, 1, [0]), (1, 16, 576, 0, [1]), (2, 16, 512, 63, [64, 0]),
    (3, 16, 576, 64, [65, 1, 128]), (5, 24, 576, 65, [0, 300, 64, 1, 127]), (4, 128, 512, 500, [10, 0, 70, 200]),
    (33, 3, 576, 1000, list(range(33))), (7, 64, 576, 4097, [1] * 7), (20, 16, 512, 700, [64 * i for i in range(20)])])
def test_shared_random(B, H, E, prefix, lens, kind):
    rng = np.random.default_rng(B * 3 + H + prefix)
    say(f"shared attention B={B} H={H} E={E} prefix={prefix} {kind}")
    run_shared(rng, B, H, E, kind, prefix, lens, E ** -0.5)


@pytest.mark.parametrize("H", [8, 64])
def test_shared_clamps_lengths_and_skips_bad_pages(H):
    rng = np.random.default_rng(5)
    say(f"shared attention, lengths outside their bound, H={H}")
    run_shared(rng, 4, H, 576, "bf16", 200, [-3, 500, 100, 129], 0.04, mpp=4, max_ctx=130)
    run_shared(rng, 3, H, 576, "fp8", 130, [100, 10, 64], 0.04, mpp=3, bad_pages=True)
    run_shared(rng, 2, H, 576, "bf16", 40, [30, 0], 0.04, bad_pages=True)   # the prefix's only page is bad


@pytest.mark.parametrize("scale", [0.0, 2.0])
def test_shared_softmax_extremes(scale):
    rng = np.random.default_rng(6)
    say(f"shared attention scale={scale}")
    run_shared(rng, 3, 40, 576, "bf16", 900, [200, 0, 64], scale, q_scale=1.0)


def test_empty_batches():
    cache = torch.zeros((2, 64, 576), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((0, 16, 576), dtype=torch.bfloat16, device="cuda")
    i0 = torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    out, lse = dsa.latent_attention_topk(q, cache, torch.zeros((1, 2), dtype=torch.int32, device="cuda"), i0, V, 1.0,
                                         seq_ids=i0[:, 0].contiguous(), want_lse=True)
    assert out.shape == (0, 16, V) and lse.shape == (0, 16)
    out, _ = dsa.latent_attention_shared(q, cache, None, 0, i0, i0[:, 0].contiguous(), V, 1.0)
    assert out.shape == (0, 16, V)
