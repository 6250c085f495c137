"""Attention over the latent cache where the softmax's reference moves in the
middle of a run of tiles, for every block size and both cache types, against
the fp64 oracle within bounds that are small next to the values (the inputs and
why they tell: latent_walk.py)."""
import numpy as np
import pytest
import torch

import dsa_lightning_indexer_03_amd as dsa
from gpu_util import say
from latent_util import V, check_attention, expect_topk
from latent_walk import assert_tight, levels, make_q, make_rows
from oracle.latent import attend

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


@pytest.mark.parametrize("kind,gain", [("bf16", 0), ("fp8", 0), ("fp8", -18), ("fp8", 12)])
@pytest.mark.parametrize("H,E", [(3, 576), (16, 576), (20, 512), (32, 576), (64, 576), (64, 512), (100, 512), (128, 576)])
def test_topk_references_move_in_one_run(H, E, kind, gain):
    """256 queries whose selections are one run of nine tiles each: in rising
    order, where references move at every tile, and for some queries falling,
    in random order and with the rising order's first tiles left out."""
    rng = np.random.default_rng(1000 + H + gain)
    T, n = 256, 566
    t, scale, rows = make_rows(rng, levels(n, 9), E, kind, gain)
    q, qv = make_q(rng, T, H, E, gain)
    idx = np.tile(np.arange(n), (T, 1))
    idx[1::8] = idx[1::8, ::-1]
    for i in range(2, T, 8):
        idx[i] = rng.permutation(n)
    idx[3::8, :130] = -1
    table = np.arange(9)[None]
    assert dsa.latent_topk_workspace_bytes(T, H, E, V, n, kind == "fp8") == 0, "more than one run"
    cache, cs = pool(t, scale, E)
    say(f"references that move, one run, H={H} E={E} {kind} gain={gain}")
    out, lse = dsa.latent_attention_topk(q.cuda(), cache, ints(table), ints(idx), V, 1.0, latent_scale=cs,
                                         seq_ids=ints(np.zeros(T)), want_lse=True)
    torch.cuda.synchronize()
    look = [0, 1, 2, 3, 4, 100, T - 1]
    pick = lambda x: x[torch.tensor(look, device=x.device)]   # noqa: E731
    want = expect_topk(qv[look], rows, table, idx[look], np.zeros(len(look), int), 1.0, 9)
    assert_tight(want, f"H={H} {kind}")
    check_attention(pick(out), pick(lse), want, f"H={H} {kind} gain={gain}")
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("kind,gain", [("bf16", 0), ("fp8", 0), ("fp8", -18)])
@pytest.mark.parametrize("B,H", [(4, 8), (2, 30), (20, 50), (128, 16)])
def test_shared_references_move_in_every_run(B, H, kind, gain):
    """A long prefix in cycles of nine tiles, cut in runs, and own keys that rise on."""
    rng = np.random.default_rng(2000 + H + gain)
    E, prefix, own = 576, 64 * 700 - 7, 200
    n_pre = -(-prefix // 64)
    lens = rng.integers(0, own, B)
    lens[0] = 0
    x = np.concatenate([levels(n_pre * 64, 9), np.tile(levels(256, 9), B)])
    t, scale, rows = make_rows(rng, x, E, kind, gain)
    q, qv = make_q(rng, B, H, E, gain)
    table = n_pre + np.arange(4 * B).reshape(B, 4)
    nbytes = dsa.latent_shared_workspace_bytes(B, H, E, V, prefix, 256, kind == "fp8")
    slots = nbytes // (B * H * 514 * 4)
    assert n_pre >= 9 * slots, f"{slots} runs: shorter than a cycle"
    cache, cs = pool(t, scale, E)
    say(f"references that move, {slots} runs, B={B} H={H} {kind} gain={gain}")
    out, lse = dsa.latent_attention_shared(q.cuda(), cache, ints(np.arange(n_pre)), prefix, ints(table), ints(lens), V,
                                           1.0, latent_scale=cs, want_lse=True)
    torch.cuda.synchronize()
    look = [0, 1, B - 1]
    want = [attend(qv[b], np.concatenate([rows[:prefix], rows[table[b, 0] * 64:table[b, 0] * 64 + lens[b]]]), 1.0, V)
            for b in look]
    pick = lambda x: x[torch.tensor(look, device=x.device)]   # noqa: E731
    assert_tight(want, f"B={B} H={H} {kind}")
    check_attention(pick(out), pick(lse), want, f"shared B={B} H={H} {kind} gain={gain}")
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
