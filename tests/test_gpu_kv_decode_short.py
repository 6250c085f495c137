"""kv_attention_decode where one wave takes a whole context: many sequences, short
contexts and selections, against the fp64 oracle; and what a call reports for its
workspace at the edges of that form."""
import numpy as np
import pytest
import torch

import dsa_lightning_indexer_03_amd as dsa
from gpu_util import say
from kv_util import ints
from oracle import kv as oracle
from test_gpu_kv_decode import case, run_and_check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H,G,longest", [(3, 4, 2, 5), (160, 8, 4, 70), (150, 40, 2, 33), (300, 48, 1, 300),
                                           (130, 3, 3, 500)])
def test_many_short_contexts(B, H, G, longest, D, kind):
    rng = np.random.default_rng(B + D)
    lens = rng.integers(0, longest + 1, B)
    lens[:4] = [longest, 0, 1, longest][:min(B, 4)]
    args, x = case(rng, [int(n) for n in lens], H, G, D, kind)
    assert dsa.kv_decode_workspace_bytes(B, H, G, D, args["block_table"].shape[1] * 64, fp8=kind == "fp8") == 0
    run_and_check(args, x, D ** -0.5, f"{B} contexts of up to {longest}, {H} heads over {G}, {D} columns, {kind}",
                  max_context_len=longest)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("K", [3, 40, 400])
def test_many_short_selections(K, kind):
    """Lists that name few positions or none, most entries outside the contexts."""
    rng = np.random.default_rng(K)
    B, G = 140, 2
    lens = [int(n) for n in rng.integers(0, 90, B)]
    idx = rng.integers(-1, 128, (B, K))
    idx[5], idx[6, 1:] = -1, 127
    args, x = case(rng, lens, 8, G, 128, kind, mpp=2, idx=idx)
    run_and_check(args, x, 0.09, f"{B} selections of {K}, {kind}", idx=idx)


def test_empty_tiles_between():
    """Tiles and rounds without a row, in front of, between and behind those with one."""
    rng = np.random.default_rng(1)
    idx = np.full((6, 900), -1)
    idx[0, 897:], idx[1, 0], idx[2, 450:460], idx[3, ::128] = [5, 6, 7], 9, np.arange(10), np.arange(8)
    idx[4] = rng.integers(0, 100, 900)
    args, x = case(rng, [100] * 6, 8, 2, 128, "bf16", mpp=2, idx=idx)
    run_and_check(args, x, 0.09, "empty tiles between", idx=idx)
    pages = np.full((2, 40), -1)                       # whole pages that are none, one with rows far behind
    args, x = case(rng, [2560, 2500], 8, 2, 64, "fp8", mpp=40)
    pages[0, 37], pages[1, 3] = x[3][0, 37], x[3][1, 3]
    args["block_table"] = ints(pages)
    run_and_check(args, x[:3] + (pages, x[4]), 0.1, "pages that are none between")


def test_bounds_of_zero():
    """No position anywhere: zeros and -inf, whatever the lengths say."""
    rng = np.random.default_rng(2)
    args, _ = case(rng, [30, 5], 4, 2, 64, "bf16")
    say("a bound of 0")
    out, lse = dsa.kv_attention_decode(**args, scale=0.1, want_lse=True, max_context_len=0)
    torch.cuda.synchronize()
    assert not bool(out.any()) and bool((lse == -float("inf")).all())
    z = {k: (v[:0] if k in ("q", "block_table", "context_lens") else v) for k, v in args.items()}
    out, lse = dsa.kv_attention_decode(**z, scale=0.1, want_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    got = oracle.decode(np.zeros((0, 4, 64)), np.zeros((1, 2, 64, 64)), np.zeros((1, 2, 64, 64)), np.zeros((0, 1)), [], 1.0)
    assert got == []
