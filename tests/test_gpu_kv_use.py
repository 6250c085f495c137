"""The write of the paged key and value caches against the oracle, and the three
operators on them as a server uses them: prompts attended and appended, then
decode steps with the indexer's selection, eager and in captured graphs."""
import numpy as np
import pytest
import torch

import dsa_lightning_indexer_03_amd as dsa
from gpu_util import say
from kv_util import bf16, check, ints
from oracle import kv as oracle
from oracle.formats import fp8_e4m3_to_f64
from oracle.kcache import encode_e4m3
from oracle.latent import U16, U32, rotate, slots

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def angles(n, R):
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, R, 2) / R)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def check_rows(cache, scale, at, G, y, err, exact, where):
    """Rows [n][G][D] at slots `at` against fp64 values y known within err; exact: bf16 inputs, columns without an error."""
    D = y.shape[2]
    pages = cache.shape[0]
    got = cache.permute(0, 2, 1, 3).reshape(pages * 64, G, D)[torch.from_numpy(at).cuda()].cpu()
    if scale is None:
        tol = np.where(err > 0, U16 * (np.abs(y) + err) + err, 0.0 if exact else U16 * np.abs(y))
        assert (np.abs(got.double().numpy() - y) <= tol).all(), where
        return
    s = scale.permute(0, 2, 1).reshape(pages * 64, G)[torch.from_numpy(at).cuda()].cpu().numpy()
    hi = (np.abs(y) + err).max(2) / 448 * (1 + 2 * U32)
    lo = np.maximum(np.abs(y) - err, 0).max(2) / 448 * (1 - 2 * U32)
    zero = (y == 0).all(2)
    lo, hi = np.where(zero, 1.0, lo), np.where(zero, 1.0, hi)
    assert ((s >= lo) & (s <= hi)).all(), f"{where}: scales"
    s = s.astype(np.float64)[..., None]
    val = fp8_e4m3_to_f64(got.numpy())
    low = fp8_e4m3_to_f64(encode_e4m3((y - err) / s - 2 * U32 * np.abs(y / s)))
    top = fp8_e4m3_to_f64(encode_e4m3((y + err) / s + 2 * U32 * np.abs(y / s)))
    assert ((val >= low) & (val <= top)).all(), f"{where}: codes"


CASES = [  # T, B, G, D, R, input, cache, pairs
    (1, 1, 8, 128, 128, "bf16", "bf16", False), (1, 1, 1, 64, 0, "f32", "fp8", False),
    (3, 2, 3, 64, 64, "f32", "bf16", True), (257, 5, 2, 128, 64, "bf16", "fp8", True),
    (130, 3, 5, 64, 16, "bf16", "bf16", False), (75, 2, 4, 128, 48, "f32", "fp8", False),
    (33, 4, 128, 64, 32, "bf16", "fp8", True), (500, 7, 1, 128, 0, "f32", "bf16", False),
    (64, 1, 16, 128, 128, "bf16", "fp8", False)]


@pytest.mark.parametrize("T,B,G,D,R,inp,kind,pairs", CASES)
def test_append_against_the_oracle(T, B, G, D, R, inp, kind, pairs):
    rng = np.random.default_rng(T * 31 + D + R)
    say(f"kv_append_rope T={T} B={B} G={G} D={D} R={R} {inp}->{kind} pairs={pairs}")
    mpp = 6
    pages = B * mpp + 2
    table = rng.permutation(pages)[: B * mpp].reshape(B, mpp).astype(np.int32)
    table[-1, -1] = pages + 5                                     # not a page of the pool
    table[0, -1] = -1
    seq = rng.integers(0, B, T).astype(np.int32)
    pos = np.zeros(T, np.int32)
    for b in range(B):                                            # distinct within each sequence, some outside
        who = np.flatnonzero(seq == b)
        pos[who] = rng.permutation(mpp * 64 + 20)[: who.size]
    if T > 2:
        seq[0], seq[1], pos[2] = -1, B, -7
    rope_len = mpp * 64 - 30                                      # the last positions have no angle
    cs = angles(rope_len, R) if R else None
    wide = rng.normal(size=(T, G, 2, D + 8)) * np.exp(rng.normal(size=(T, G, 1, 1)))   # strided tokens and heads
    if T > 5:
        wide[5] = 0
    src, val = bf16(wide) if inp == "bf16" else (torch.from_numpy(wide.astype(np.float32)),
                                                 wide.astype(np.float32).astype(np.float64))
    src = src.cuda()
    k, v = src[:, :, 0, :D], src[:, :, 1, :D]
    size = 2 if kind == "bf16" else 1
    raw = [torch.from_numpy(rng.integers(0, 120, size=(pages, G, 64, D * size)).astype(np.uint8)).cuda() for _ in "kv"]
    caches = [x.clone().view(torch.bfloat16) if kind == "bf16" else x.clone() for x in raw]
    scale0 = torch.rand((pages, G, 64), device="cuda")
    scales = [scale0.clone() if kind == "fp8" else None for _ in "kv"]
    dsa.kv_append_rope(k, v, ints(seq), ints(pos), ints(table), *caches,
                       cos_sin=None if cs is None else torch.from_numpy(cs).cuda(), k_scale=scales[0],
                       v_scale=scales[1], interleaved=pairs)
    torch.cuda.synchronize()
    at = slots(seq, pos, table, pages, rope_len if R else None)
    live = at >= 0
    at = at[live]
    y = val[live, :, 0, :D]
    err = np.zeros_like(y)
    if R:
        n = y.shape[0]
        turn = np.repeat(cs[pos[live]], G, 0)
        y, err = rotate(y.reshape(n * G, D), turn, 0, pairs)
        y, err = y.reshape(n, G, D), err.reshape(n, G, D)
    check_rows(caches[0], scales[0], at, G, y, err, inp == "bf16", "keys")
    y = val[live, :, 1, :D]
    check_rows(caches[1], scales[1], at, G, y, np.zeros_like(y), inp == "bf16", "values")
    other = np.ones(pages * 64, bool)
    other[at] = False
    other = torch.from_numpy(other).cuda()
    for c, r in zip(caches, raw):
        a, b = (x.view(torch.uint8).view(pages, G, 64, -1).permute(0, 2, 1, 3).reshape(pages * 64, -1)[other] for x in (c, r))
        assert torch.equal(a, b)
    for s in scales:
        if s is not None:
            a, b = (x.permute(0, 2, 1).reshape(pages * 64, G)[other] for x in (s, scale0))
            assert torch.equal(a, b)


def test_append_what_is_not_finite():
    """NaNs stay NaNs and do not enter a row's scale; infinities stay themselves; the rows beside them are as without."""
    T, G, D = 6, 2, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((T, G, D), generator=g, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    seq, pos, table = ints(np.zeros(T)), ints(np.arange(T)), ints([[0]])
    kw = lambda: dict(k_cache=torch.zeros((1, G, 64, D), dtype=torch.uint8, device="cuda"),    # noqa: E731
                      v_cache=torch.zeros((1, G, 64, D), dtype=torch.uint8, device="cuda"),
                      k_scale=torch.zeros((1, G, 64), device="cuda"), v_scale=torch.zeros((1, G, 64), device="cuda"))
    say("rows that are not finite")
    a, b = kw(), kw()
    dsa.kv_append_rope(k, v, seq, pos, table, **a)
    k2, v2 = k.clone(), v.clone()
    k2[2, 1, 7], v2[3, 0, 100], v2[3, 0, 101] = float("nan"), float("inf"), -float("inf")
    dsa.kv_append_rope(k2, v2, seq, pos, table, **b)
    torch.cuda.synchronize()
    kb = b["k_cache"].view(torch.float8_e4m3fn).float()
    assert bool(kb[0, 1, 2, 7].isnan()) and int(kb.isnan().sum()) == 1
    keep = torch.ones((1, G, 64, D), dtype=torch.bool, device="cuda")
    keep[0, 1, 2] = False
    assert torch.equal(a["k_cache"][keep], b["k_cache"][keep])
    rest = k2[2, 1].float()
    rest[7] = 0
    assert float(b["k_scale"][0, 1, 2]) == float(np.float32(rest.abs().max().item()) / np.float32(448))
    vb = b["v_cache"].view(torch.float8_e4m3fn).float() * b["v_scale"][..., None]
    assert float(vb[0, 0, 3, 100]) == float("inf") and float(vb[0, 0, 3, 101]) == -float("inf")
    keep = torch.ones((1, G, 64, D), dtype=torch.bool, device="cuda")
    keep[0, 0, 3] = False
    assert torch.equal(a["v_cache"][keep], b["v_cache"][keep])


def test_append_nothing_and_far():
    """No tokens: a no-op.  The last page of pools past 2^32 bytes."""
    G, D, pages = 8, 128, 34000
    z = torch.zeros((0, G, D), dtype=torch.bfloat16, device="cuda")
    one = torch.ones((2, G, 64, D), dtype=torch.bfloat16, device="cuda")
    dsa.kv_append_rope(z, z, ints([]), ints([]), ints([[0]]), one, one.clone())
    kc, vc = (torch.empty((pages, G, 64, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    kc[0], vc[0] = 3, 4
    k, v = (torch.randn((64, G, D), device="cuda").bfloat16() for _ in "kv")
    say("append into the last pages of two 4.4 GB pools")
    dsa.kv_append_rope(k, v, ints(np.zeros(64)), ints(np.arange(64)), ints([[pages - 1]]), kc, vc)
    torch.cuda.synchronize()
    assert bool((one == 1).all())
    assert torch.equal(kc[-1], k.transpose(0, 1)) and torch.equal(vc[-1], v.transpose(0, 1))
    assert bool((kc[0] == 3).all()) and bool((vc[0] == 4).all())


class Server:
    """Caches of B sequences and the indexer's key cache beside them, one block table."""

    def __init__(self, kind, B=3, mpp=8, H=8, G=2, D=128, seed=0):
        self.rng = np.random.default_rng(seed)
        self.kind, self.B, self.H, self.G, self.D = kind, B, H, G, D
        self.pages = B * mpp + 1
        self.table = self.rng.permutation(self.pages)[:B * mpp].reshape(B, mpp)
        bf = kind == "bf16"
        fill = float("nan") if bf else 0x7F
        self.caches = [torch.full((self.pages, G, 64, D), fill, dtype=torch.bfloat16 if bf else torch.uint8,
                                  device="cuda") for _ in "kv"]
        self.scales = [None if bf else torch.full((self.pages, G, 64), float("nan"), device="cuda") for _ in "kv"]
        self.kc = torch.zeros((self.pages, 64, 128), dtype=torch.uint8, device="cuda")
        self.ks = torch.zeros((self.pages, 64), device="cuda")
        self.cs = torch.from_numpy(angles(64 * mpp, D)).cuda()

    def append(self, seq, pos, k, v, ik):
        dsa.kv_append_rope(k, v, seq, pos, ints(self.table), *self.caches, cos_sin=self.cs, k_scale=self.scales[0],
                           v_scale=self.scales[1])
        dsa.kcache_append(ik, seq, pos, ints(self.table), self.kc, self.ks)

    def values(self):
        got = []
        for c, s in zip(self.caches, self.scales):
            x = c.double() if s is None else c.view(torch.float8_e4m3fn).double() * s.double()[..., None]
            got.append(x.cpu().numpy())
        return got


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_prompt_then_decode(kind):
    """Prompts attended whole (keys rotated by the caller) and appended; then decode
    steps: append one token a sequence, select with the indexer, attend over the
    selection and over everything."""
    sv = Server(kind)
    B, H, G, D, lens = sv.B, sv.H, sv.G, sv.D, np.array([3, 130, 301])
    T = int(lens.sum()) + 5                                    # five padding rows
    cu = np.concatenate([[0], np.cumsum(lens)])
    seq = np.append(np.repeat(np.arange(B), lens), [-1] * 5)
    pos = np.append(np.concatenate([np.arange(n) for n in lens]), [0] * 5)
    qkv, val = bf16(sv.rng.normal(size=(T, (H + 2 * G) * D)))
    qkv = qkv.cuda()
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([H * D, G * D, G * D], 1))
    qv, kvv, vvv = (x.reshape(T, -1, D) for x in np.split(val, [H * D, (H + G) * D], 1))
    out, lse = dsa.prompt_attention(q, k, v, ints(cu), D ** -0.5, want_lse=True)
    torch.cuda.synchronize()
    check(out, lse, list(zip(*oracle.prompt(qv, kvv, vvv, cu, D ** -0.5))), f"prompts, {kind}")
    sv.append(ints(seq), ints(pos), k, v, torch.randn((T, 128), device="cuda").bfloat16())
    K = 96
    for step in range(3):
        say(f"decode step {step} {kind}")
        new = lambda *s: bf16(sv.rng.normal(size=s))[0].cuda()   # noqa: E731
        sv.append(ints(np.append(np.arange(B), -1)), ints(np.append(lens, 0)), new(B + 1, G, D), new(B + 1, G, D),
                  new(B + 1, 128))
        lens = lens + 1
        idx, _ = dsa.indexer_decode_paged(new(B, 16, 128), torch.rand((B, 16), device="cuda"), sv.kc, sv.ks,
                                          ints(sv.table), ints(lens), K)
        q, qv = bf16(1.5 * sv.rng.normal(size=(B, H, D)))
        kw = dict(k_scale=sv.scales[0], v_scale=sv.scales[1], want_lse=True)
        some = dsa.kv_attention_decode(q.cuda(), *sv.caches, ints(sv.table), ints(lens), D ** -0.5, topk_idx=idx, **kw)
        every = dsa.kv_attention_decode(q.cuda(), *sv.caches, ints(sv.table), ints(lens), D ** -0.5, **kw)
        torch.cuda.synchronize()
        rows = sv.values()
        got = idx.cpu().numpy()
        check(*some, oracle.decode(qv, *rows, sv.table, lens, D ** -0.5, idx=got), f"selected, step {step}")
        check(*every, oracle.decode(qv, *rows, sv.table, lens, D ** -0.5), f"every position, step {step}")


def test_graphs():
    """Append and both forms of the decode step captured twice, the second graph
    with its own workspace, replayed with inputs that change and eager calls of the
    same kind between the replays."""
    sv = [Server("fp8", mpp=40, seed=s) for s in (3, 4)]
    B, H, G, D, K = 3, 8, 2, 128, 700
    held, graphs = [], []
    for i, s in enumerate(sv):
        n = 2500
        for b in range(B):
            r = lambda *z: torch.randn(z, device="cuda").bfloat16()   # noqa: E731
            s.append(ints(np.full(n, b)), ints(np.arange(n)), r(n, G, D), r(n, G, D), r(n, 128))
        h = dict(k=torch.zeros((4, G, D), device="cuda", dtype=torch.bfloat16), seq=ints([0, 1, 2, -1]),
                 pos=ints([0, 0, 0, 4]), table=ints(s.table), idx=ints(np.zeros((B, K))), n=ints([1, 2, 1]),
                 q=torch.zeros((B, H, D), device="cuda", dtype=torch.bfloat16))
        h["ws"] = torch.empty(dsa.kv_decode_workspace_bytes(B, H, G, D, 2560, fp8=True) + 16, dtype=torch.uint8,
                              device="cuda")

        def step(h, s, own):
            dsa.kv_append_rope(h["k"], h["k"], h["seq"], h["pos"], h["table"], *s.caches, cos_sin=s.cs,
                               k_scale=s.scales[0], v_scale=s.scales[1])
            kw = dict(k_scale=s.scales[0], v_scale=s.scales[1], want_lse=True)
            a = dsa.kv_attention_decode(h["q"], *s.caches, h["table"], h["n"], 0.1, topk_idx=h["idx"], **kw)
            b = dsa.kv_attention_decode(h["q"], *s.caches, h["table"], h["n"], 0.1, workspace=h["ws"] if own else None,
                                        **kw)
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
        for h in held:
            h["k"].copy_(bf16(rng.normal(size=(4, G, D)))[0])
            h["q"].copy_(bf16(1.5 * rng.normal(size=(B, H, D)))[0])
            h["pos"].copy_(ints(rng.integers(0, 2500, 4)))
            h["n"].copy_(ints(rng.integers(0, 2501, B)))
            h["idx"].copy_(ints(rng.integers(-1, 2500, (B, K))))
        for graph in graphs:                       # both in flight before anything waits
            graph.replay()
        for h, s in zip(held, sv):
            want = step(h, s, False)               # eager, on the same inputs
            torch.cuda.synchronize()
            for j, (a, b) in enumerate(zip(h["out"], want)):
                assert torch.equal(a, b), f"replay {replay}, result {j}"
