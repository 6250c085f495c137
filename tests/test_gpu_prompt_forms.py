"""Every form of prompt_attention (128 rows and one key group with tiles
of 64 and of 32 keys, or two groups, 64 rows and four groups) against the fp64
oracle, and against each other's results where the heads of a call only change
its form."""
import numpy as np
import pytest
import torch

import dsa_lightning_indexer_03_amd as dsa
from gpu_util import say
from kv_util import bf16, check, ints
from oracle import kv as oracle

pytestmark = pytest.mark.gpu
DIMS = [(64, 64), (128, 128), (192, 128)]
# lengths, heads, key/value heads: one group (short or many), two groups, four groups
FORMS = {"one": ([90, 33, 0, 120, 64], 12, 2), "one, many blocks": ([300] * 3 + [1], 120, 1),
         "one, longer": ([1300, 900], 44, 2), "one, long": ([2200, 2150], 24, 3),
         "two": ([700], 64, 2), "two, ragged": ([900, 130, 0, 1100], 24, 3),
         "four": ([200, 191], 8, 2), "four, one head": ([1100, 65, 129], 1, 1), "four, long": ([2100], 16, 1)}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(rng, T, H, G, D, V):
    return zip(*(bf16(s * rng.normal(size=(T, n, w))) for s, n, w in ((1.5, H, D), (1, G, D), (1, G, V))))


@pytest.mark.parametrize("D,V", DIMS)
@pytest.mark.parametrize("form", FORMS)
def test_against_the_oracle(form, D, V):
    """Rows around every tile's and block's edge, and some of the others."""
    lens, H, G = FORMS[form]
    rng = np.random.default_rng(len(form) + D)
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1]) + 7
    t, x = make(rng, T, H, G, D, V)
    say(f"{form}: prompts of {lens}, {H} heads over {G}, {D} columns")
    out, lse = dsa.prompt_attention(*(y.cuda() for y in t), ints(cu), D ** -0.5, want_lse=True)
    torch.cuda.synchronize()
    assert not bool(out[cu[-1]:].any()) and bool((lse[cu[-1]:] == -float("inf")).all())
    assert bool(out.isfinite().all()) and bool(lse[:cu[-1]].isfinite().all())
    rows, want = [], []
    for a, b in zip(cu, cu[1:]):
        edge = [i for i in range(a, b) if (i - a + 2) % 32 <= 3 or i == b - 1 or rng.random() < 0.05]
        rows += edge
        want += [oracle.grouped(x[0][i], x[1][a:i + 1], x[2][a:i + 1], D ** -0.5) for i in edge]
    check(out[rows], lse[rows], want, form)


@pytest.mark.parametrize("D,V", DIMS)
@pytest.mark.parametrize("form", FORMS)
def test_what_a_row_does_not_see(form, D, V):
    """Values that are not finite in a row of each 32 of the last sequence: rows before
    it get what they get without, bit for bit; the others get it."""
    lens, H, G = FORMS[form]
    rng = np.random.default_rng(3)
    cu = np.concatenate([[0], np.cumsum(lens)])
    a, b = int(cu[-2]), int(cu[-1])
    t, _ = make(rng, b, H, G, D, V)
    q, k, v = (y.cuda() for y in t)
    say(f"{form}: values that are not finite, {D} columns")
    want, wl = dsa.prompt_attention(q, k, v, ints(cu), 0.1, want_lse=True)
    for at in sorted({a, a + (b - a) // 3, max(a, b - 40), b - 1}):
        for bad in (float("inf"), float("nan")):
            w = v.clone()
            w[at, G - 1, 9] = bad
            got, gl = dsa.prompt_attention(q, k, w, ints(cu), 0.1, want_lse=True)
            torch.cuda.synchronize()
            seen = torch.zeros_like(got, dtype=torch.bool)
            seen[at:b, (G - 1) * (H // G):, 9] = True
            assert torch.equal(got[~seen], want[~seen]) and torch.equal(gl, wl), f"{bad} at {at}"
            assert not bool(got[seen].isfinite().any()), f"{bad} at {at}"


@pytest.mark.parametrize("form", FORMS)
def test_far_scores(form):
    """Scores of size 2^40: a row's highest takes everything, whichever key group has
    it.  Keys are -1, 0 or 1 in one column, so that scores are exact."""
    lens, H, G = FORMS[form]
    rng = np.random.default_rng(4)
    cu = np.concatenate([[0], np.cumsum(lens)])
    T, D = int(cu[-1]), 128
    sign = rng.integers(0, 3, T) - 1.0
    k = torch.zeros((T, G, D), dtype=torch.bfloat16, device="cuda")
    k[:, :, 0] = torch.from_numpy(sign).cuda().bfloat16()[:, None]
    q = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 2.0 ** 40
    v, vv = bf16(rng.normal(size=(T, G, D)))
    say(f"{form}: scores of 2^40")
    out, lse = dsa.prompt_attention(q, k, v.cuda(), ints(cu), 1.0, want_lse=True)
    torch.cuda.synchronize()
    out, lse = out[:, 0].double().cpu().numpy(), lse[:, 0].double().cpu().numpy()
    for a, b in zip(cu, cu[1:]):
        for i in range(a, b, 7):
            top = sign[a:i + 1].max()
            who = np.flatnonzero(sign[a:i + 1] == top) + a
            # equal probabilities: one rounding of them, common to all, and the output's; fp32 sums
            tol = np.abs(vv[a:i + 1, 0]).max(0) * (2.0 ** -7 + (i - a + 20) * 2.0 ** -24)
            assert (np.abs(out[i] - vv[who, 0].mean(0)) <= tol).all(), i
            assert abs(lse[i] - (top * 2.0 ** 40 + np.log(len(who)))) <= 2.0 ** -22 * (abs(top) * 2.0 ** 40 + 9), i


@pytest.mark.parametrize("form", FORMS)
def test_the_same_call_twice(form):
    lens, H, G = FORMS[form]
    rng = np.random.default_rng(6)
    cu = ints(np.concatenate([[0], np.cumsum(lens)]))
    t, _ = make(rng, sum(lens), H, G, 128, 128)
    t = [y.cuda() for y in t]
    say(f"{form}: repeated calls")
    first = dsa.prompt_attention(*t, cu, 0.1, want_lse=True)
    for _ in range(4):
        again = dsa.prompt_attention(*t, cu, 0.1, want_lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("B,longest", [(64, 5), (65, 300), (4095, 2), (4096, 3), (5000, 1), (300000, 1)])
def test_as_many_sequences_as_rows(B, longest):
    """Sequences found 64 places at a time, in one to four steps; empty ones among them."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, longest + 1, B)
    lens[[0, B // 2, B - 1]] = longest
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1]) + 130
    t, x = make(rng, T, 2, 1, 64, 64)
    say(f"{B} sequences of up to {longest} rows")
    out, lse = dsa.prompt_attention(*(y.cuda() for y in t), ints(cu), 0.125, want_lse=True)
    torch.cuda.synchronize()
    assert not bool(out[cu[-1]:].any()) and bool((lse[cu[-1]:] == -float("inf")).all())
    if longest == 1:
        assert torch.equal(out[:cu[-1]].cpu(), t[2][:cu[-1]].expand(-1, 2, -1))
    some = [b for b in np.r_[0:70, rng.integers(0, B, 60), max(0, B - 70):B] if b < B]
    rows, want = [], []
    for b in sorted(set(some)):
        for i in range(cu[b], cu[b + 1]):
            rows.append(i)
            want.append(oracle.grouped(x[0][i], x[1][cu[b]:i + 1], x[2][cu[b]:i + 1], 0.125))
    check(out[rows], lse[rows], want, f"{B} sequences")
