"""The inputs of latent_walk.py tell a right walk over the keys from one whose
sums do not follow a reference that moves: on the CPU, with the mistakes
planted in the walk."""
import numpy as np
import pytest
import torch

from latent_util import V, check_attention
from latent_walk import assert_tight, levels, make_q, make_rows, walk
from oracle.latent import attend


def case(kind, H, gain, n=566, cycle=9):
    rng = np.random.default_rng(1000 + H + gain)
    _, scale, rows = make_rows(rng, levels(n, cycle), 576, kind, gain)
    return make_q(rng, 1, H, 576, gain)[1][0], rows, None if scale is None else scale.numpy()


@pytest.mark.parametrize("kind,gain", [("bf16", 0), ("fp8", 0), ("fp8", -18), ("fp8", 12)])
@pytest.mark.parametrize("H", [16, 20, 40])
@pytest.mark.parametrize("step", [32, 64])
def test_planted_mistakes_show(kind, gain, H, step):
    q, rows, scales = case(kind, H, gain)
    want = [attend(q, rows, 1.0, V)]
    assert_tight(want, f"H={H} {kind}")

    def passes(plant, block):
        out, lse = walk(q, rows, scales, 1.0, step, block, plant)
        try:
            check_attention(torch.from_numpy(out)[None], torch.from_numpy(lse)[None], want, "walk")
            return True
        except AssertionError:
            return False
    for block in (16, 64):   # rows whose references move together: a wave's, or a workgroup's
        assert passes(None, block)
        for plant in ("sums", "outputs", "both"):
            assert not passes(plant, block), plant


def test_the_cycle_repeats():
    """Levels of a long list: every run of more than a cycle's tiles sees references rise."""
    x = levels(64 * 20, 9)
    assert x[0] == 0 and x[63] < 1 and x[64 * 8] == 8 and x[64 * 9] == 0 and x.max() < 9
