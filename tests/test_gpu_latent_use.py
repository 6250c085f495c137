"""The operators on the two caches as a server uses them: one after another on
one pool, on other streams, in captured graphs, with the caller's workspaces,
in pools past 2^32 bytes; and the same call twice."""
import numpy as np
import pytest
import torch

import dsa_lightning_indexer_03_amd as dsa
from gpu_util import say
from latent_util import V, bf16, check_attention, expect_topk, make_pool
from oracle.latent import attend, slots

pytestmark = pytest.mark.gpu
E, H, SCALE = 576, 16, 576 ** -0.5


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def angles(n, R=64):
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, R, 2) / R)
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()


def values(latent, scale):
    """fp64 rows of a device cache."""
    x = latent.view(torch.float8_e4m3fn) if latent.dtype == torch.uint8 else latent
    x = x.double() if scale is None else x.double() * scale.double()[..., None]
    return x.view(-1, latent.shape[2]).cpu().numpy()


class Server:
    """Caches of B sequences that start with the same `prefix` positions."""

    def __init__(self, kind, B=3, mpp=8, prefix=128, seed=0):
        self.rng = np.random.default_rng(seed)
        self.kind, self.B, self.prefix = kind, B, prefix
        self.pages = prefix // 64 + B * mpp + 1
        perm = self.rng.permutation(self.pages)
        self.ptab = perm[: prefix // 64]
        self.own = perm[prefix // 64:prefix // 64 + B * mpp].reshape(B, mpp)
        self.table = np.concatenate([np.tile(self.ptab, (B, 1)), self.own], 1)
        if kind == "bf16":
            self.latent = torch.full((self.pages, 64, E), float("nan"), dtype=torch.bfloat16, device="cuda")
            self.ls = None
        else:
            self.latent = torch.full((self.pages, 64, E), 0x7F, dtype=torch.uint8, device="cuda")
            self.ls = torch.full((self.pages, 64), float("nan"), device="cuda")
        self.kc = torch.zeros((self.pages, 64, 128), dtype=torch.uint8, device="cuda")
        self.ks = torch.zeros((self.pages, 64), device="cuda")
        self.cs = angles(64 * self.table.shape[1])

    def append(self, seq, pos):
        T = len(seq)
        new = bf16(self.rng.normal(size=(T, E + 128)))[0].cuda()
        dsa.cache_append_rope(new[:, :E], ints(seq), ints(pos), ints(self.table), self.latent, self.cs,
                              latent_scale=self.ls, index_k=new[:, E:], k_cache=self.kc, k_scale=self.ks)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_append_then_index_then_attend(kind):
    """Prompt rows appended (the shared prefix once), then decode steps: append
    one token a sequence, select positions with the indexer, attend over them."""
    sv = Server(kind)
    B, K, lens = sv.B, 96, np.array([3, 130, 301])
    sv.append(np.zeros(sv.prefix, int), np.arange(sv.prefix))
    sv.append(np.repeat(np.arange(B), lens), np.concatenate([sv.prefix + np.arange(n) for n in lens]))
    for step in range(3):
        say(f"decode step {step} {kind}")
        sv.append(np.append(np.arange(B), [-1, 0]), np.append(sv.prefix + lens, [5, -1]))   # two padding rows
        lens = lens + 1
        qi = bf16(sv.rng.normal(size=(B, 16, 128)))[0].cuda()
        w = torch.rand((B, 16), device="cuda")
        idx, _ = dsa.indexer_decode_paged(qi, w, sv.kc, sv.ks, ints(sv.table), ints(sv.prefix + lens), K)
        q, qv = bf16(1.5 * sv.rng.normal(size=(B, H, E)))
        out, lse = dsa.latent_attention_topk(q.cuda(), sv.latent, ints(sv.table), idx, V, SCALE,
                                             latent_scale=sv.ls, want_lse=True)
        every = np.full((B, sv.prefix + lens.max()), -1)
        for b in range(B):
            every[b, : sv.prefix + lens[b]] = np.arange(sv.prefix + lens[b])
        out_e, lse_e = dsa.latent_attention_topk(q.cuda(), sv.latent, ints(sv.table), ints(every), V, SCALE,
                                                 latent_scale=sv.ls, want_lse=True)
        out_s, lse_s = dsa.latent_attention_shared(q.cuda(), sv.latent, ints(sv.ptab), sv.prefix, ints(sv.own),
                                                   ints(lens), V, SCALE, latent_scale=sv.ls, want_lse=True)
        torch.cuda.synchronize()
        rows, got = values(sv.latent, sv.ls), idx.cpu().numpy()
        assert all(((got[b] >= 0) == (np.arange(K) < sv.prefix + lens[b])).all() and
                   got[b].max() < sv.prefix + lens[b] for b in range(B))

        def want(ids):
            s = [slots(np.full(ids.shape[1], b), ids[b], sv.table, sv.pages) for b in range(B)]
            return [attend(qv[b], rows[s[b][s[b] >= 0]], SCALE, V) for b in range(B)]
        check_attention(out, lse, want(got), f"selected, step {step}")
        check_attention(out_e, lse_e, want(every), f"every position, step {step}")
        check_attention(out_s, lse_s, want(every), f"prefix and own, step {step}")


def inputs(seed, T, K, mpp=12, heads=H):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = T * mpp
    return dict(q=torch.randn((T, heads, E), generator=g, device="cuda", dtype=torch.bfloat16),
                latent_cache=torch.randn((pages, 64, E), generator=g, device="cuda", dtype=torch.bfloat16),
                block_table=torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32).view(T, mpp),
                topk_idx=torch.randint(-1, mpp * 64, (T, K), generator=g, device="cuda", dtype=torch.int32))


def shared_args(x, n):
    T, mpp = x["block_table"].shape
    return dict(q=x["q"], latent_cache=x["latent_cache"], prefix_table=x["block_table"][0].contiguous(),
                prefix_len=64 * mpp - 5, block_table=x["block_table"], context_lens=n)


@pytest.mark.parametrize("heads", [16, 24, 64, 128])
def test_the_same_call_twice(heads):
    """Splits over workgroups and their joins do not depend on the order of execution."""
    x = inputs(1, 9, 700, heads=heads)
    n = ints(np.arange(9) * 70)
    say(f"repeated calls, {heads} heads")
    first = [dsa.latent_attention_topk(**x, v_dim=V, scale=SCALE, want_lse=True),
             dsa.latent_attention_shared(**shared_args(x, n), v_dim=V, scale=SCALE, want_lse=True)]
    for _ in range(5):
        again = [dsa.latent_attention_topk(**x, v_dim=V, scale=SCALE, want_lse=True),
                 dsa.latent_attention_shared(**shared_args(x, n), v_dim=V, scale=SCALE, want_lse=True)]
        for a, b in zip(first, again):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("T,heads,K", [(23, 97, 400), (11, 100, 129), (40, 55, 300)])
def test_many_rows_in_several_parts(T, heads, K, kind):
    """Enough rows that a wave joins each, in parts that some rows do not reach."""
    rng = np.random.default_rng(T)
    mpp, pages = 4, 4 * T
    table = rng.permutation(pages).reshape(T, mpp)
    idx = rng.integers(-1, mpp * 64, (T, K))
    idx[1], idx[2, 64:], idx[3, : K - 2] = -1, -1, -1
    cache, scale, rows = make_pool(rng, pages, E, kind)
    q, qv = bf16(1.5 * rng.normal(size=(T, heads, E)))
    say(f"{T} queries of {heads} heads, {K} selected, {kind}")
    out, lse = dsa.latent_attention_topk(q.cuda(), cache, ints(table), ints(idx), V, SCALE, latent_scale=scale,
                                         want_lse=True)
    torch.cuda.synchronize()
    check_attention(out, lse, expect_topk(qv, rows, table, idx, np.arange(T), SCALE, pages), "many rows")


def test_two_streams():
    """Calls on two streams at once, each with inputs made on its own stream."""
    xs = [inputs(2 + i, 40, 1000) for i in range(2)]
    want = [dsa.latent_attention_topk(**x, v_dim=V, scale=SCALE)[0] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    say("two streams")
    for turn in range(4):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                mine = {k: v.clone() for k, v in x.items()}
                got.append(dsa.latent_attention_topk(**mine, v_dim=V, scale=SCALE)[0])
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for g, w in zip(got, want):
            assert torch.equal(g, w), f"turn {turn}"


def test_graphs():
    """Append, selection's attention and shared attention captured twice, the
    second graph with its own workspaces, replayed with inputs that change and
    eager calls of the same kind between the replays."""
    sv = [Server("fp8", seed=s) for s in (3, 4)]
    B, K, T = 3, 700, 5
    held, graphs = [], []
    for i, s in enumerate(sv):
        g = torch.Generator(device="cuda").manual_seed(i)
        h = dict(new=torch.zeros((T, E + 128), device="cuda", dtype=torch.bfloat16), seq=ints([0, 1, 2, -1, 1]),
                 pos=ints([0, 0, 0, 4, 1]), table=ints(s.table), own=ints(s.own), ptab=ints(s.ptab),
                 idx=ints(np.zeros((B, K))), n=ints([1, 2, 1]),
                 q=torch.zeros((B, H, E), device="cuda", dtype=torch.bfloat16))
        s.append(np.zeros(s.prefix, int), np.arange(s.prefix))
        for b in range(B):
            s.append(np.full(300, b), s.prefix + np.arange(300))

        h["ws1"] = torch.empty(dsa.latent_topk_workspace_bytes(B, H, E, V, K, True) + 16, dtype=torch.uint8,
                               device="cuda")
        h["ws2"] = torch.empty(dsa.latent_shared_workspace_bytes(B, H, E, V, s.prefix, 512, True) + 16,
                               dtype=torch.uint8, device="cuda")

        def step(h, s, own_space):
            dsa.cache_append_rope(h["new"][:, :E], h["seq"], h["pos"], h["table"], s.latent, s.cs, latent_scale=s.ls,
                                  index_k=h["new"][:, E:], k_cache=s.kc, k_scale=s.ks)
            a = dsa.latent_attention_topk(h["q"], s.latent, h["table"], h["idx"], V, SCALE, latent_scale=s.ls,
                                          want_lse=True, workspace=h["ws1"] if own_space else None)
            b = dsa.latent_attention_shared(h["q"], s.latent, h["ptab"], s.prefix, h["own"], h["n"], V, SCALE,
                                            latent_scale=s.ls, want_lse=True, workspace=h["ws2"] if own_space else None)
            return a + b

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(h, s, i == 1)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            h["out"] = step(h, s, i == 1)
        held.append(h)
        graphs.append(graph)
    rng = np.random.default_rng(5)
    for replay in range(4):
        say(f"replay {replay}")
        for h, s in zip(held, sv):
            h["new"].copy_(bf16(rng.normal(size=(T, E + 128)))[0])
            h["q"].copy_(bf16(1.5 * rng.normal(size=(B, H, E)))[0])
            h["pos"].copy_(ints([s.prefix + replay, s.prefix + 7, s.prefix + 2 * replay, 4, s.prefix + 8]))
            h["n"].copy_(ints(rng.integers(0, 301, B)))
            h["idx"].copy_(ints(rng.integers(-1, s.prefix + 300, (B, K))))
        for graph in graphs:                       # both in flight before anything waits
            graph.replay()
        for h, s in zip(held, sv):
            want = step(h, s, False)               # eager, on the same inputs
            torch.cuda.synchronize()
            for k, (a, b) in enumerate(zip(h["out"], want)):
                assert torch.equal(a, b), f"replay {replay}, result {k}"


def test_the_callers_workspace():
    x = inputs(6, 4, 600)
    want, _ = dsa.latent_attention_topk(**x, v_dim=V, scale=SCALE)
    n = dsa.latent_topk_workspace_bytes(4, H, E, V, 600)
    assert n > 0
    ws = torch.full((n + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    got, _ = dsa.latent_attention_topk(**x, v_dim=V, scale=SCALE, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and bool((ws[n:] == 0xAB).all())
    with pytest.raises(ValueError, match="workspace"):
        dsa.latent_attention_topk(**x, v_dim=V, scale=SCALE, workspace=ws.cpu())
    with pytest.raises(ValueError, match="workspace"):
        dsa.latent_attention_topk(**x, v_dim=V, scale=SCALE, workspace=ws[::2])


def test_refusals_on_the_device():
    x = inputs(7, 2, 64)
    call = lambda **kw: dsa.latent_attention_topk(**{**x, **kw}, v_dim=V, scale=SCALE)   # noqa: E731
    wide = torch.zeros((2, H, 2 * E), device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="contiguous"):
        call(q=wide[:, :, :E])
    shifted = torch.zeros(2 * H * E + 8, device="cuda", dtype=torch.bfloat16)[4:4 + 2 * H * E].view(2, H, E)
    with pytest.raises(Exception, match="align"):
        call(q=shifted)
    with pytest.raises(ValueError, match="one row per query"):
        call(block_table=x["block_table"][:1].contiguous())
    with pytest.raises(ValueError, match="backward"):
        call(q=x["q"].clone().requires_grad_())
    with torch.no_grad():
        call(q=x["q"].clone().requires_grad_())
    with pytest.raises(ValueError, match="latent_scale"):
        call(latent_scale=torch.ones((24, 64), device="cuda"))
    with pytest.raises(ValueError, match="device"):
        call(topk_idx=x["topk_idx"].cpu())
    with pytest.raises(ValueError, match="must be in"):
        dsa.latent_attention_shared(x["q"], x["latent_cache"], x["block_table"][0].contiguous(), 2 ** 32 + 5,
                                    x["block_table"], ints([1, 1]), V, SCALE)
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("heads", [16, 24, 64, 128])
def test_pool_beyond_32_bit_offsets(heads, kind):
    """Rows whose byte offsets pass 2^32, in the pool's last pages."""
    pages = 73000 if kind == "bf16" else 140000
    say(f"attention on the last pages of a 5 GB pool, {heads} heads, {kind}")
    cache = torch.empty((pages, 64, E), dtype=torch.bfloat16 if kind == "bf16" else torch.uint8, device="cuda")
    scale = None
    if kind == "fp8":
        scale = torch.full((pages, 64), 0.02, device="cuda")
    rng = np.random.default_rng(8)
    x = bf16(rng.normal(size=(4 * 64, E)))[0].cuda()
    if kind == "fp8":
        x = (x.float() * 20).to(torch.float8_e4m3fn).view(torch.uint8)
    small = x.view(4, 64, E)
    cache[-4:] = small
    q = bf16(rng.normal(size=(2, heads, E)))[0].cuda()
    idx = ints(rng.integers(-1, 128, (2, 150)))
    high, low = ints(pages - 4 + np.arange(4).reshape(2, 2)), ints(np.arange(4).reshape(2, 2))
    s4 = None if scale is None else scale[:4].contiguous()
    pre_h, pre_l, n = ints(pages - 4 + np.arange(2)), ints(np.arange(2)), ints([64, 100])
    got = [dsa.latent_attention_topk(q, cache, high, idx, V, SCALE, latent_scale=scale)[0],
           dsa.latent_attention_shared(q, cache, pre_h, 100, high, n, V, SCALE, latent_scale=scale)[0]]
    want = [dsa.latent_attention_topk(q, small, low, idx, V, SCALE, latent_scale=s4)[0],
            dsa.latent_attention_shared(q, small, pre_l, 100, low, n, V, SCALE, latent_scale=s4)[0]]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and bool(a.any()) for a, b in zip(got, want))


@pytest.mark.parametrize("heads", [1, 24, 64, 128])
@pytest.mark.parametrize("K", [1, 3])
def test_one_fp8_row_rounds_once(heads, K):
    """A query whose only row (K times) is an fp8 row gets that row, rounded
    once.  The product of its probability and scale is 1 up to the rounding of
    the exponent: scores in base 2 stay below 64 here, so the exponent is off by
    2^-18 at most, the product by 2^-18, and bf16 rounds it to 1; the sum, which
    is not rounded, keeps that error.  What is left is the output's half step,
    2^-8, those 2^-18, and a few roundings of fp32, 2^-20 together."""
    rng = np.random.default_rng(heads + K)
    T = 40
    cache, scale, rows = make_pool(rng, 2 * T, E, "fp8")
    scale *= torch.exp(torch.randn(scale.shape, device="cuda"))
    rows = values(cache, scale)
    table = ints(np.arange(2 * T).reshape(T, 2))
    at = rng.integers(0, 128, T)
    q = bf16(rng.normal(size=(T, heads, E)))[0].cuda()
    assert np.abs(np.einsum("the,te->th", q.double().cpu().numpy(), rows[np.arange(T) * 128 + at])).max() * SCALE < 44
    say(f"one fp8 row {K} times, {heads} heads")
    out, _ = dsa.latent_attention_topk(q, cache, table, ints(np.tile(at[:, None], (1, K))), V, SCALE, latent_scale=scale)
    torch.cuda.synchronize()
    want = rows[np.arange(T) * 128 + at][:, None, :V]
    assert (np.abs(out.double().cpu().numpy() - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -18 + 2.0 ** -20)).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("heads", [7, 20, 100])
def test_long_lists_of_keys(heads, kind):
    """Selections and prefixes of many thousand rows, in 32 parts each, the last
    ones short; every part holds keys of its own."""
    rng = np.random.default_rng(heads)
    mpp, T, K = 330, 2, 20001
    pages = mpp + 1
    cache, scale, rows = make_pool(rng, pages, E, kind)
    table = rng.permutation(pages)[:mpp]
    idx = np.stack([rng.permutation(mpp * 64)[:K] for _ in range(T)])
    q, qv = bf16(1.5 * rng.normal(size=(T, heads, E)))
    say(f"{K} selected rows and a prefix of {mpp * 64 - 3}, {heads} heads, {kind}")
    out, lse = dsa.latent_attention_topk(q.cuda(), cache, ints(np.tile(table, (T, 1))), ints(idx), V, SCALE,
                                         latent_scale=scale, want_lse=True)
    n = mpp * 64 - 3
    own = np.full((T, 1), mpp)                         # the page that no table held: not an id of the pool for query 1
    own[1] = pages
    out_s, lse_s = dsa.latent_attention_shared(q.cuda(), cache, ints(table), n, ints(own), ints([0, 9]), V, SCALE,
                                               latent_scale=scale, want_lse=True)
    torch.cuda.synchronize()
    check_attention(out, lse, expect_topk(qv, rows, np.tile(table, (T, 1)), idx, np.arange(T), SCALE, pages), "selected")
    s = slots(np.zeros(n, int), np.arange(n), table[None], pages)
    check_attention(out_s, lse_s, [attend(qv[b], rows[s], SCALE, V) for b in range(T)], "prefix")
