"""GPU parity of prompt_attention against the fp64 oracle: every head shape,
packed sequences of lengths around the tiles and blocks, strided rows, values
that masked rows must not meet, scores far from zero."""
import numpy as np
import pytest
import torch

import dsa_lightning_indexer_03_amd as dsa
from gpu_util import say
from kv_util import bf16, check, ints
from oracle import kv as oracle

pytestmark = pytest.mark.gpu
DIMS = [(64, 64), (128, 128), (192, 128)]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def cu_of(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def make(rng, T, H, G, D, V, size=1.5):
    q, qv = bf16(size * rng.normal(size=(T, H, D)))
    k, kv = bf16(rng.normal(size=(T, G, D)))
    v, vv = bf16(rng.normal(size=(T, G, V)))
    return (q.cuda(), k.cuda(), v.cuda()), (qv, kv, vv)


def run_and_check(t, x, lens, scale, where):
    cu = cu_of(lens)
    say(where)
    out, lse = dsa.prompt_attention(*t, ints(cu), scale, want_lse=True)
    torch.cuda.synchronize()
    o, l, eo, el = oracle.prompt(*x, cu, scale)
    check(out, lse, list(zip(o, l, eo, el)), where)
    assert not bool(out[cu[-1]:].any())
    return out, lse


LENS = [[1], [2], [31, 1, 33], [63, 64, 65], [127], [128], [129, 0, 1], [0, 300, 0], [200, 191, 5]]


@pytest.mark.parametrize("D,V", DIMS)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_lengths(lens, D, V):
    rng = np.random.default_rng(sum(lens) + D)
    t, x = make(rng, sum(lens) + 3, 4, 2, D, V)
    run_and_check(t, x, lens, D ** -0.5, f"prompts of {lens}, {D} and {V} columns")


@pytest.mark.parametrize("D,V", DIMS)
@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (5, 5), (7, 7), (8, 1), (16, 2), (14, 2), (128, 4), (24, 8)])
def test_heads(H, G, D, V):
    rng = np.random.default_rng(H * G + D)
    lens = [37, 96, 150] if H < 64 else [37, 90]
    t, x = make(rng, sum(lens), H, G, D, V)
    run_and_check(t, x, lens, D ** -0.5, f"{H} heads over {G}, {D} and {V} columns")


@pytest.mark.parametrize("n", [63, 64, 65, 130, 700])
def test_many_sequences(n):
    """Sequences counted in one pass (up to 63 and the rows behind them) or in several."""
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 5, n)
    lens[rng.integers(0, n, 3)] = [130, 1, 257]
    t, x = make(rng, int(lens.sum()) + 140, 2, 1, 64, 64)
    run_and_check(t, x, lens, 0.125, f"{n} sequences")


def test_no_sequence_has_rows():
    rng = np.random.default_rng(5)
    t, _ = make(rng, 200, 3, 3, 128, 128)
    say("rows of no sequence only")
    out, lse = dsa.prompt_attention(*t, ints([0, 0, 0]), 0.1, want_lse=True)
    torch.cuda.synchronize()
    assert not bool(out.any()) and bool((lse == -float("inf")).all())
    z = [x[:0] for x in t]
    out, lse = dsa.prompt_attention(*z, ints([0, 0]), 0.1, want_lse=True)
    assert out.shape == (0, 3, 128) and lse.shape == (0, 3)


@pytest.mark.parametrize("D,V", DIMS)
def test_strided_rows(D, V):
    """Rows cut out of one projection, out of [heads, tokens, columns], and one head for all."""
    rng = np.random.default_rng(D)
    T, H, G, lens = 170, 6, 2, [100, 70]
    both, val = bf16(rng.normal(size=(T, H * D + G * D + G * V + 8)))
    both = both.cuda()
    cut = lambda a: (a[:, :H * D].reshape(T, H, D), a[:, H * D:(H + G) * D].reshape(T, G, D),   # noqa: E731
                     a[:, (H + G) * D:(H + G) * D + G * V].reshape(T, G, V))
    t = (both[:, :H * D].view(T, H, D), both[:, H * D:(H + G) * D].view(T, G, D),
         both[:, (H + G) * D:(H + G) * D + G * V].view(T, G, V))
    first = run_and_check(t, cut(val), lens, 0.1, f"rows of one projection, {D}")
    turned = tuple(x.transpose(0, 1).contiguous().transpose(0, 1) for x in t)
    assert turned[0].stride(1) != D
    again = run_and_check(turned, cut(val), lens, 0.1, f"heads first, {D}")
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    one = (t[0], t[1][:, :1].expand(T, G, D), t[2][:, :1].expand(T, G, V))
    x = cut(val)
    run_and_check(one, (x[0], np.repeat(x[1][:, :1], G, 1), np.repeat(x[2][:, :1], G, 1)), lens, 0.1, f"broadcast, {D}")


@pytest.mark.parametrize("scale", [-0.1, 0.0, 0.7, 1e-30])
def test_scales(scale):
    rng = np.random.default_rng(7)
    t, x = make(rng, 150, 2, 2, 128, 128)
    run_and_check(t, x, [140], scale, f"scale {scale}")


@pytest.mark.parametrize("D,V", DIMS)
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_what_a_row_does_not_see(bad, D, V):
    """Values and keys that are not finite, in rows that earlier rows of the same
    tile, other sequences and other heads do not see: those get what they get
    without them, bit for bit; rows that see such a value get it."""
    rng = np.random.default_rng(11)
    lens, H, G = [150, 70], 4, 2
    t, x = make(rng, 260, H, G, D, V)
    cu = ints(cu_of(lens))
    say(f"{bad} in rows that others do not see, {D}")
    want, wl = dsa.prompt_attention(*t, cu, 0.1, want_lse=True)
    at = 133                                     # of the first sequence, inside its last tile
    v = t[2].clone()
    v[at, 0, 5] = bad
    v[220:] = bad                                # rows of no sequence
    k = t[1].clone()
    k[220:] = bad
    got, gl = dsa.prompt_attention(t[0], k, v, cu, 0.1, want_lse=True)
    torch.cuda.synchronize()
    seen = torch.zeros_like(got, dtype=torch.bool)
    seen[at:150, :2, 5] = True
    assert torch.equal(got[~seen], want[~seen]) and torch.equal(gl, wl)
    if bad == bad:
        assert bool((got[seen].float() == bad).all())
    else:
        assert bool(got[seen].isnan().all())
    k = t[1].clone()
    k[at, 1, 3] = float("nan")                   # rows from here on: NaN; the ones before: as they were
    q = t[0].clone()
    q[20, 3] = float("nan")                      # one head of one row
    got, gl = dsa.prompt_attention(q, k, t[2], cu, 0.1, want_lse=True)
    torch.cuda.synchronize()
    hit = torch.zeros(got.shape[:2], dtype=torch.bool, device="cuda")
    hit[at:150, 2:] = True
    hit[20, 3] = True
    assert bool(got[hit].isnan().all()) and bool(gl[hit].isnan().all())
    assert torch.equal(got[~hit], want[~hit]) and torch.equal(gl[~hit], wl[~hit])


@pytest.mark.parametrize("D,V", DIMS)
def test_infinities_of_both_signs(D, V):
    """+inf and -inf seen together are NaN; alone they are themselves."""
    rng = np.random.default_rng(12)
    t, _ = make(rng, 64, 1, 1, D, V)
    v = t[2].clone()
    v[40, 0, 1], v[50, 0, 1], v[45, 0, 2] = float("inf"), -float("inf"), -float("inf")
    say(f"infinities of both signs, {D}")
    out, _ = dsa.prompt_attention(t[0], t[1], v, ints([0, 64]), 0.1)
    torch.cuda.synchronize()
    out = out[:, 0].float()
    assert bool(out[:40].isfinite().all()) and bool((out[40:50, 1] == float("inf")).all())
    assert bool(out[50:, 1].isnan().all()) and bool((out[45:, 2] == -float("inf")).all())
    assert bool(out[:, 3:].isfinite().all())


@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 40])
def test_far_scores(size):
    """Scores of size 2^20 and 2^40, far past their rounding: a row's highest score
    takes everything.  Keys are +-1 in one column, so that scores are exact: row i's
    highest are its rows with the larger key."""
    T, D = 200, 128
    rng = np.random.default_rng(1)
    sign = rng.integers(0, 3, T) - 1.0
    k = torch.zeros((T, 1, D), dtype=torch.bfloat16, device="cuda")
    k[:, 0, 0] = torch.from_numpy(sign).cuda().bfloat16()
    q = torch.zeros((T, 1, D), dtype=torch.bfloat16, device="cuda")
    q[:, 0, 0] = size
    v, vv = bf16(rng.normal(size=(T, 1, D)))
    say(f"scores of {size}")
    out, lse = dsa.prompt_attention(q, k, v.cuda(), ints([0, T]), 1.0, want_lse=True)
    torch.cuda.synchronize()
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for i in range(T):
        top = sign[:i + 1].max()
        mean = vv[:i + 1, 0][sign[:i + 1] == top].mean(0)
        # equal probabilities: one rounding of them, common to all, and the output's; fp32 sums
        tol = np.abs(vv[:i + 1, 0]).max(0) * (2.0 ** -8 + 2.0 ** -8 + (i + 20) * 2.0 ** -24)
        assert (np.abs(out[i, 0] - mean) <= tol).all(), i
        n = (sign[:i + 1] == top).sum()
        assert abs(lse[i, 0] - (top * size + np.log(n))) <= 2.0 ** -22 * (abs(top * size) + np.log(n) + 1), i


def test_one_row_rounds_once():
    """A row that sees itself only gets its value."""
    rng = np.random.default_rng(9)
    t, x = make(rng, 130, 4, 4, 192, 128)
    say("sequences of one row")
    out, _ = dsa.prompt_attention(*t, ints(np.arange(131)), 0.1)
    torch.cuda.synchronize()
    assert torch.equal(out, t[2])


def test_again_streams_and_graphs():
    """The same call twice; two streams at once; two captured graphs replayed with
    inputs that change, eager calls between the replays."""
    rng = np.random.default_rng(21)
    xs = [make(rng, 900, 8, 2, 128, 128)[0] for _ in range(2)]
    cus = [ints(cu_of([500, 17, 380])), ints(cu_of([3, 890]))]
    want = [dsa.prompt_attention(*x, c, 0.1, want_lse=True) for x, c in zip(xs, cus)]
    again = [dsa.prompt_attention(*x, c, 0.1, want_lse=True) for x, c in zip(xs, cus)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, g in zip(want, again) for a, b in zip(w, g))
    streams = [torch.cuda.Stream() for _ in range(2)]
    say("two streams")
    for _ in range(3):
        got = []
        for x, c, s in zip(xs, cus, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                mine = [y.clone() for y in x]
                got.append(dsa.prompt_attention(*mine, c, 0.1, want_lse=True))
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))
    graphs, outs = [], []
    for x, c in zip(xs, cus):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(dsa.prompt_attention(*x, c, 0.1, want_lse=True))
        graphs.append(g)
    for replay in range(3):
        say(f"replay {replay}")
        for x, c in zip(xs, cus):
            for y in x:
                y.copy_(torch.randn_like(y))
            c.copy_(ints(cu_of([100 + replay, 790, 3])) if len(c) == 4 else ints(cu_of([700 - replay, 100])))
        for g in graphs:
            g.replay()
        for x, c, o in zip(xs, cus, outs):
            w = dsa.prompt_attention(*x, c, 0.1, want_lse=True)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_long_prompt_spot_rows():
    """20000 rows; the oracle takes some of them."""
    rng = np.random.default_rng(31)
    lens, H, G, D = [13001, 6990], 4, 2, 128
    t, x = make(rng, 19991, H, G, D, D)
    say("prompts of 13001 and 6990 rows")
    out, lse = dsa.prompt_attention(*t, ints(cu_of(lens)), D ** -0.5, want_lse=True)
    torch.cuda.synchronize()
    at = [0, 63, 64, 127, 128, 5000, 12927, 12928, 13000, 13001, 13065, 19000, 19990]
    want = []
    for i in at:
        a = 0 if i < 13001 else 13001
        want.append(oracle.grouped(x[0][i], x[1][a:i + 1], x[2][a:i + 1], D ** -0.5))
    check(out[at], lse[at], want, "long prompts")


def test_rows_beyond_32_bit_offsets():
    """Rows whose element offsets pass 2^31: 131072 tokens of 128 heads, in short sequences."""
    T, H, G, D = 131072 + 64, 128, 128, 192
    say("131136 tokens, 128 heads of 192")
    q = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
    k, v = torch.empty_like(q), torch.empty((T, G, 128), dtype=torch.bfloat16, device="cuda")
    for y in (q, k, v):
        y.normal_()
    cu = list(range(0, T + 1, 64))
    out, lse = dsa.prompt_attention(q, k, v, ints(cu), 0.07, want_lse=True)
    small = [y[-128:].contiguous() for y in (q, k, v)]
    want, wl = dsa.prompt_attention(*small, ints([0, 64, 128]), 0.07, want_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(out[-128:], want) and torch.equal(lse[-128:], wl)


def test_refusals_on_the_device():
    rng = np.random.default_rng(3)
    (q, k, v), _ = make(rng, 10, 4, 2, 128, 128)
    cu = ints([0, 10])
    wide = torch.zeros((10, 4, 256), device="cuda", dtype=torch.bfloat16)
    for bad, match in [((wide[:, :, ::2], k, v, cu), "contiguous"), ((q, k[:9], v, cu), "must be"),
                       ((q, k, v, cu.long()), "cu_seqlens"), ((q, k, v, cu[:1]), "cu_seqlens"),
                       ((q, k, v, cu.cpu()), "device"), ((q, k.cpu(), v, cu), "device"),
                       ((q.requires_grad_(), k, v, cu), "backward")]:
        with pytest.raises(ValueError, match=match):
            dsa.prompt_attention(*bad, 0.1)
    with torch.no_grad():
        dsa.prompt_attention(q, k, v, cu, 0.1)
    q = q.detach()
    for bad in [(q[:, :, :64], k[:, :, :64], v, cu), (q[:, :3], k, v, cu),
                (torch.zeros(10 * 512 + 8, device="cuda", dtype=torch.bfloat16)[4:4 + 5120].view(10, 4, 128), k, v, cu)]:
        with pytest.raises(Exception, match="status"):
            dsa.prompt_attention(*bad, 0.1)
    torch.cuda.synchronize()
