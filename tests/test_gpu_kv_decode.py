"""GPU parity of kv_attention_decode against the fp64 oracle: cache types, head
shapes, context lengths around tiles, pages and runs, selections, slots and
pages that hold nothing, scores far from zero, workspaces, streams, graphs."""
import numpy as np
import pytest
import torch

import dsa_lightning_indexer_03_amd as dsa
from gpu_util import say
from kv_util import bf16, check, ints, make_pool
from oracle import kv as oracle

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "fp8"]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def case(rng, lens, H, G, D, kind, mpp=None, idx=None, size=1.5):
    """Caches of len(lens) sequences, NaN wherever no sequence has a position (with a
    selection: where none is selected)."""
    B = len(lens)
    mpp = mpp or max(1, -(-max(lens) // 64))
    pages = B * mpp + 2
    table = rng.permutation(pages)[:B * mpp].reshape(B, mpp)
    live = np.zeros((pages, 64), bool)
    for b in range(B):
        pos = np.arange(lens[b]) if idx is None else oracle.positions(idx[b], lens[b])
        page, slot = oracle.place(pos, table[b], pages)
        live[page, slot] = True
    kc, ks, kv = make_pool(rng, pages, G, D, kind, live)
    vc, vs, vv = make_pool(rng, pages, G, D, kind, live)
    q, qv = bf16(size * rng.normal(size=(B, H, D)))
    args = dict(q=q.cuda(), k_cache=kc, v_cache=vc, block_table=ints(table), context_lens=ints(lens), k_scale=ks,
                v_scale=vs, topk_idx=None if idx is None else ints(idx))
    return args, (qv, kv, vv, table, lens)


def run_and_check(args, x, scale, where, idx=None, **kw):
    say(where)
    out, lse = dsa.kv_attention_decode(**args, scale=scale, want_lse=True, **kw)
    torch.cuda.synchronize()
    check(out, lse, oracle.decode(*x, scale, idx=idx), where)
    return out, lse


LENS = [[1], [0, 2, 31], [32, 33, 63, 64, 65], [127, 128, 129, 0], [255, 256, 257, 300], [1000, 3, 511, 513]]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_lengths(lens, D, kind):
    rng = np.random.default_rng(sum(lens) + D)
    args, x = case(rng, lens, 8, 2, D, kind)
    run_and_check(args, x, D ** -0.5, f"contexts of {lens}, {D} columns, {kind}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G", [(1, 1), (5, 5), (7, 1), (16, 1), (17, 1), (32, 1), (33, 1), (64, 1), (65, 1), (128, 1),
                                 (128, 128), (40, 2), (24, 3)])
def test_heads(H, G, D, kind):
    rng = np.random.default_rng(H * G + D)
    args, x = case(rng, [150, 0, 77], H, G, D, kind)
    run_and_check(args, x, D ** -0.5, f"{H} heads over {G}, {D} columns, {kind}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,G", [(8, 2), (20, 1), (48, 1)])
@pytest.mark.parametrize("K", [1, 31, 33, 200, 700])
def test_selections(K, H, G, kind):
    """Lists in any order, with -1, positions outside the context, positions twice, none at all."""
    rng = np.random.default_rng(K + H)
    lens = [500, 40, 0, 640, 1]
    idx = rng.integers(-1, 700, (5, K))
    idx[3] = -1
    args, x = case(rng, lens, H, G, 128, kind, mpp=10, idx=idx)
    run_and_check(args, x, 0.09, f"{K} selected, {H} heads over {G}, {kind}", idx=idx)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
def test_long_contexts_in_runs(D, kind):
    """Contexts cut over workgroups, the last run short; a bound far above the lengths."""
    rng = np.random.default_rng(D)
    lens = [9001, 130, 0, 4096]
    args, x = case(rng, lens, 6, 2, D, kind)
    assert dsa.kv_decode_workspace_bytes(4, 6, 2, D, 9001, fp8=kind == "fp8") > 0
    a = run_and_check(args, x, D ** -0.5, f"long contexts, {D} columns, {kind}", max_context_len=9001)
    run_and_check(args, x, D ** -0.5, f"long contexts, the table's bound, {D} columns, {kind}")
    # a bound below a length cuts that context
    x = x[:4] + ([5000, 130, 0, 4096],)
    b = run_and_check(args, x, D ** -0.5, f"a bound of 5000, {D} columns, {kind}", max_context_len=5000)
    assert not torch.equal(a[0][0], b[0][0])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("topk", [False, True])
def test_pages_that_are_none(kind, topk):
    """Page ids outside the pool are pages without rows: in the middle, at the end, all of a sequence's."""
    rng = np.random.default_rng(4)
    lens = [300, 300, 64, 200]
    idx = rng.permutation(300)[None].repeat(4, 0)[:, :150] if topk else None
    args, x = case(rng, lens, 8, 2, 128, kind, idx=idx)
    table = x[3].copy()
    table[0, 2], table[1, 4], table[2], table[3, 0] = -1, 1 << 20, -(1 << 31), x[1].shape[0]
    args["block_table"] = ints(table)
    run_and_check(args, x[:3] + (table, lens), 0.1, f"pages that are none, {kind}", idx=idx)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-30])
def test_scales(scale):
    rng = np.random.default_rng(7)
    args, x = case(rng, [150, 20], 4, 2, 64, "bf16")
    run_and_check(args, x, scale, f"scale {scale}")


@pytest.mark.parametrize("kind", KINDS)
def test_a_head_that_is_not_finite(kind):
    """A query head with NaN or infinities leaves the heads beside it as they are."""
    rng = np.random.default_rng(8)
    args, _ = case(rng, [700, 90], 8, 1, 128, kind)
    say(f"a head that is not finite, {kind}")
    want = dsa.kv_attention_decode(**args, scale=0.1, want_lse=True)
    for bad in (float("nan"), float("inf")):
        q = args["q"].clone()
        q[0, 3, 7], q[1, 0] = bad, bad
        got = dsa.kv_attention_decode(**{**args, "q": q}, scale=0.1, want_lse=True)
        torch.cuda.synchronize()
        keep = torch.ones((2, 8), dtype=torch.bool, device="cuda")
        keep[0, 3] = keep[1, 0] = False
        for a, b in zip(got, want):
            assert torch.equal(a[keep], b[keep]) and not bool(a[~keep].isfinite().all())


@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 40])
def test_far_scores(size):
    """Scores far past their rounding: the highest ones take everything, across waves and runs."""
    rng = np.random.default_rng(1)
    n, D = 3000, 128
    args, x = case(rng, [n], 4, 1, D, "bf16")
    sign = rng.integers(0, 3, args["k_cache"].shape[0] * 64).reshape(-1, 64) - 1.0
    args["k_cache"].zero_()
    args["k_cache"][:, 0, :, 0] = torch.from_numpy(sign).cuda().bfloat16()
    q = torch.zeros((1, 4, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = torch.tensor([size, -size, size / 2, 0.0]).cuda().bfloat16()
    args["q"] = q
    say(f"scores of {size}")
    out, lse = dsa.kv_attention_decode(**args, scale=1.0, want_lse=True)
    torch.cuda.synchronize()
    page, slot = oracle.place(np.arange(n), x[3][0], x[1].shape[0])
    s, v = sign[page, slot], x[2][page, 0, slot]
    for h, f in enumerate([size, -size, size / 2, 0.0]):
        top = (s * f).max()
        who = s * f == top
        # equal probabilities: one rounding of them, common to all, and the output's; fp32 sums
        tol = np.abs(v).max(0) * (2.0 ** -8 + 2.0 ** -8 + (n + 20) * 2.0 ** -24)
        assert (np.abs(out[0, h].double().cpu().numpy() - v[who].mean(0)) <= tol).all()
        want = top + np.log(who.sum())
        assert abs(float(lse[0, h]) - want) <= 2.0 ** -22 * (abs(top) + np.log(n) + 1)


@pytest.mark.parametrize("heads", [1, 8, 24, 64])
@pytest.mark.parametrize("K", [1, 3])
def test_one_fp8_row_rounds_once(heads, K):
    """A query whose only row (K times) is an fp8 row gets that row, rounded once:
    its probability times its scale, in units of that scale, is 1 up to fp32
    roundings (scores in base 2 stay below 64, so the exponent is off by 2^-18 at
    most), which bf16 rounds to 1.  What is left is the output's half step, 2^-8,
    the sum's 2^-18, and a few roundings of fp32, 2^-20 together."""
    rng = np.random.default_rng(heads + K)
    B = 20
    idx = np.tile(rng.integers(0, 128, B)[:, None], (1, K))
    args, x = case(rng, [128] * B, heads, 1, 128, "fp8", idx=idx, size=1.0)
    f = torch.exp(torch.randn(args["v_scale"].shape, device="cuda"))
    args["v_scale"] *= f
    say(f"one fp8 row {K} times, {heads} heads")
    out, _ = dsa.kv_attention_decode(**args, scale=128 ** -0.5)
    torch.cuda.synchronize()
    page, slot = x[3][np.arange(B), idx[:, 0] // 64], idx[:, 0] % 64
    codes = args["v_cache"].view(torch.float8_e4m3fn).double().cpu().numpy()[page, 0, slot]
    want = codes * args["v_scale"].double().cpu().numpy()[page, 0, slot][:, None]
    want = want[:, None]
    assert (np.abs(out.double().cpu().numpy() - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -18 + 2.0 ** -20)).all()


def big(seed, B=5, n=3000, H=8, G=2, kind="bf16", K=None):
    rng = np.random.default_rng(seed)
    idx = None if K is None else rng.integers(-1, n, (B, K))
    args, _ = case(rng, [n - 7 * b for b in range(B)], H, G, 128, kind, idx=idx)
    return args


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K", [None, 1500])
def test_again_and_streams(K, kind):
    """Runs and their join do not depend on the order of execution; two streams at once."""
    xs = [big(i, kind=kind, K=K) for i in range(2)]
    say(f"again and on two streams, {kind}, {K}")
    want = [dsa.kv_attention_decode(**x, scale=0.1, want_lse=True) for x in xs]
    for _ in range(3):
        got = [dsa.kv_attention_decode(**x, scale=0.1, want_lse=True) for x in xs]
        assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                mine = {k: None if v is None else v.clone() for k, v in x.items()}
                got.append(dsa.kv_attention_decode(**mine, scale=0.1, want_lse=True))
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))


def test_the_callers_workspace():
    """The caller's scratch: its contents on entry do not matter, nothing behind its end is written."""
    x = big(3)
    want, wl = dsa.kv_attention_decode(**x, scale=0.1, want_lse=True)
    n = dsa.kv_decode_workspace_bytes(5, 8, 2, 128, x["block_table"].shape[1] * 64)
    assert n > 0
    for fill in (0x7F, 0xFF):
        ws = torch.full((n + 64,), fill, dtype=torch.uint8, device="cuda")
        got, gl = dsa.kv_attention_decode(**x, scale=0.1, want_lse=True, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(gl, wl) and bool((ws[n:] == fill).all())
    with pytest.raises(ValueError, match="workspace"):
        dsa.kv_attention_decode(**x, scale=0.1, workspace=ws.cpu())


def test_pool_beyond_32_bit_offsets():
    """Rows whose byte offsets pass 2^32, in the pools' last pages."""
    pages, G, D = 34000, 8, 128
    say("attention on the last pages of two 4.4 GB pools")
    kc = torch.empty((pages, G, 64, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    kc[-4:].normal_()
    vc[-4:].normal_()
    q = torch.randn((2, 16, D), device="cuda").bfloat16()
    high, low, n = ints(pages - 4 + np.arange(4).reshape(2, 2)), ints(np.arange(4).reshape(2, 2)), ints([100, 128])
    idx = ints(np.random.default_rng(0).integers(-1, 128, (2, 70)))
    for i in (None, idx):
        got = dsa.kv_attention_decode(q, kc, vc, high, n, 0.1, topk_idx=i)[0]
        want = dsa.kv_attention_decode(q, kc[-4:].contiguous(), vc[-4:].contiguous(), low, n, 0.1, topk_idx=i)[0]
        torch.cuda.synchronize()
        assert torch.equal(got, want) and bool(got.any())


def test_refusals_on_the_device():
    x = big(9, B=2, n=100)
    call = lambda **kw: dsa.kv_attention_decode(**{**x, **kw}, scale=0.1)   # noqa: E731
    for kw, match in [(dict(q=x["q"][:, :, :64]), "G and D|contiguous"), (dict(q=x["q"].float()), "q must be"),
                      (dict(block_table=x["block_table"][:1]), "shape"), (dict(context_lens=x["context_lens"].long()), "context_lens"),
                      (dict(topk_idx=ints([[1]])), "topk_idx"), (dict(topk_idx=torch.zeros((2, 0), dtype=torch.int32, device="cuda")), "topk_idx"),
                      (dict(k_scale=torch.ones((4, 2, 64), device="cuda")), "k_scale"), (dict(max_context_len=-1), "max_context_len"),
                      (dict(v_cache=x["v_cache"][:-1]), "caches|k_cache"), (dict(v_cache=x["v_cache"].cpu()), "device"),
                      (dict(q=x["q"].clone().requires_grad_()), "backward")]:
        with pytest.raises(ValueError, match=match):
            call(**kw)
    with pytest.raises(Exception, match="status"):
        call(max_context_len=1 << 20)
    with pytest.raises(Exception, match="status"):
        call(q=x["q"][:, :7].contiguous())
    torch.cuda.synchronize()


def test_two_graphs_on_one_workspace():
    """Two captured steps with one scratch between them, replayed one after another."""
    xs = [big(i, K=k) for i, k in ((5, None), (6, 1500))]
    n = max(dsa.kv_decode_workspace_bytes(5, 8, 2, 128, x["block_table"].shape[1] * 64, k) for x, k in zip(xs, (0, 1500)))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for x in xs:
        dsa.kv_attention_decode(**x, scale=0.1, want_lse=True, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(dsa.kv_attention_decode(**x, scale=0.1, want_lse=True, workspace=ws))
        graphs.append(g)
    for replay in range(3):
        say(f"replay {replay} of two graphs on one workspace")
        for x in xs:
            x["q"].copy_(torch.randn_like(x["q"]))
        for g in graphs:
            g.replay()
        for x, o in zip(xs, outs):
            want = dsa.kv_attention_decode(**x, scale=0.1, want_lse=True)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(o, want))
