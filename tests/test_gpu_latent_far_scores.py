"""Scores far beyond any that a model makes, but finite: the highest one holds
all the weight, as in any softmax whose scores are rounded before their maximum
is taken off."""
import numpy as np
import pytest
import torch

import dsa_lightning_indexer_03_amd as dsa
from gpu_util import say
from latent_util import V

pytestmark = pytest.mark.gpu
E = 576


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("H", [5, 16, 30, 64, 128])
@pytest.mark.parametrize("power,scale", [(20, 1.0), (33, 1.0), (40, -0.7), (60, 0.3), (100, 1.0)])
def test_far_scores(H, power, scale, kind):
    """Scores of some 2^power: the product of a query's one column with that of
    each row.  Those columns are 1 .. 2 in bf16 or E4M3 steps of 2^-3, so the
    highest score is above the others by 2^-4 of itself, 2^16 at least, and the
    weight of its rows, which are alike, is 1 to the last bit."""
    rng = np.random.default_rng(H + power)
    T, n = 3, 500
    value = rng.integers(-8, 9, size=(n, E)).astype(np.float32) / 8
    value[:, V:] = 0
    value[:, V] = 1 + rng.integers(0, 8, n) / 8.0
    best = value[:, V].max() if scale > 0 else value[:, V].min()
    value[value[:, V] == best, :V] = value[np.argmax(value[:, V] == best), :V]
    t = torch.from_numpy(value)
    t = torch.cat([t, t[: -n % 64]]).view(-1, 64, E).cuda()
    cache, cs = (t.bfloat16(), None) if kind == "bf16" else (t.to(torch.float8_e4m3fn).view(torch.uint8),
                                                            torch.ones(t.shape[:2], device="cuda"))
    q = torch.zeros((T, H, E), dtype=torch.bfloat16, device="cuda")
    lead = torch.from_numpy(1 + rng.integers(0, 128, size=(T, H)) / 128.0).cuda() * 2.0 ** power
    q[:, :, V] = lead.bfloat16()
    idx = np.stack([rng.permutation(n) for _ in range(T)])
    say(f"scores of 2^{power}, H={H} scale={scale} {kind}")
    out, lse = dsa.latent_attention_topk(q, cache, ints(np.arange(8)[None]), ints(idx), V, scale, latent_scale=cs,
                                         seq_ids=ints(np.zeros(T)), want_lse=True)
    lens, prefix = ints([n - 64] * T), 64
    out2, lse2 = dsa.latent_attention_shared(q, cache, ints([0]), prefix, ints(np.tile(np.arange(1, 8), (T, 1))), lens,
                                             V, scale, latent_scale=cs, want_lse=True)
    torch.cuda.synchronize()
    row = torch.from_numpy(value[np.argmax(value[:, V] == best), :V]).double()
    top = scale * best * q[:, :, V].double().cpu() + np.log((value[:, V] == best).sum())
    for o, l in ((out, lse), (out2, lse2)):
        o, l = o.double().cpu(), l.double().cpu()
        # one rounding of P and one of the output
        assert bool(((o - row).abs() <= 2 * 2.0 ** -8 * row.abs()).all()), "out is not the row of the highest score"
        assert bool(((l - top).abs() <= 2.0 ** -21 * top.abs()).all()), "lse"


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("T,H,n", [(2, 16, 500), (260, 16, 500), (2, 31, 300), (260, 64, 300), (3, 64, 500), (2, 128, 500)])
def test_a_bad_head_stays_alone(T, H, n, kind):
    """A head whose query holds NaN or infinities gives NaN, in one run and in
    several; the heads beside it, in its block and its wave, what they give without."""
    g = torch.Generator(device="cuda").manual_seed(T + H)
    x = torch.randn((8, 64, E), generator=g, device="cuda")
    cache, cs = (x.bfloat16(), None) if kind == "bf16" else ((x * 100).clamp(-448, 448).to(torch.float8_e4m3fn),
                                                            0.005 + 0.01 * torch.rand((8, 64), generator=g, device="cuda"))
    q = torch.randn((T, H, E), generator=g, device="cuda").bfloat16()
    idx = torch.randint(0, 512, (T, n), generator=g, device="cuda", dtype=torch.int32)
    say(f"bad heads, T={T} H={H} {kind}")

    def call(q):
        return dsa.latent_attention_topk(q, cache, ints(np.arange(8)[None]), idx, V, 0.04, latent_scale=cs,
                                         seq_ids=ints(np.zeros(T)), want_lse=True)
    want, wl = call(q)
    bad = torch.zeros((T, H), dtype=torch.bool, device="cuda")
    bad[0, 1], bad[T - 1, 0], bad[1, H - 1] = True, True, True
    q[0, 1, 100], q[T - 1, 0, 550], q[1, H - 1, 7] = float("nan"), float("nan"), float("inf")
    out, lse = call(q)
    torch.cuda.synchronize()
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], wl[~bad])
    assert bool(torch.isnan(out[bad]).all()) and not bool(torch.isfinite(lse[bad]).any())
