"""Cases for the operators around the indexer in a sparse-attention layer: the caches' write path with the position
rotation, attention over the selected latent rows, and attention of a batch that shares a long prefix.

The latent cache holds one E-wide row per token (a compressed key, whose first V columns are the value too), in pages of
64 tokens; every head of a query reads the same rows."""
import math
import random

import torch

_dsa = None  # the package, imported on the first call that needs it
own = False

PAGE = 64
V = 512       # value columns of a latent row
D = 128       # index key width
ROPE = 64     # rotated columns
E4M3_MAX = 448.0

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one new token of one sequence: a decode step's write, launch latency alone
        dict(name="append, 1 token", op="append", tokens=1, seqs=1, E=576, input="bf16", cache="bf16", index=True,
             kv_pairs=True, index_pairs=False),
        # a decode step of a full serving batch, fp8 latent rows
        dict(name="append, 128 tokens, fp8", op="append", tokens=128, seqs=128, E=576, input="bf16", cache="fp8",
             index=True, kv_pairs=True, index_pairs=False),
        # a prompt chunk over ragged sequences, fp32 projections, rows without a separate rotary part
        dict(name="append, 4099 tokens, f32", op="append", tokens=4099, seqs=7, E=512, input="f32", cache="fp8",
             index=False, kv_pairs=False, index_pairs=False),
        # the largest prompt the indexer's headline workload prefills, both caches in one call
        dict(name="append, 32768 tokens", op="append", tokens=32768, seqs=3, E=576, input="bf16", cache="bf16",
             index=True, kv_pairs=True, index_pairs=False),

        # one query after the indexer's selection of 2048 positions, heads split over 8 GPUs: latency
        dict(name="topk, 1 query, 16 heads", op="topk", seqs=1, rows=1, pad=0, H=16, K=2048, E=576, lo=32768, hi=32768,
             cache="bf16"),
        # a serving batch's decode step: 64 queries with contexts of their own, rows gathered from a large cache
        dict(name="topk, 64 queries, 16 heads", op="topk", seqs=64, rows=1, pad=0, H=16, K=2048, E=576, lo=4096,
             hi=32768, cache="bf16"),
        # odd batch, head count and selection, fp8 rows, short contexts that leave slots of the selection empty
        dict(name="topk, 37 queries, 24 heads, fp8", op="topk", seqs=37, rows=1, pad=0, H=24, K=1000, E=512, lo=0,
             hi=6000, cache="fp8"),
        # a prompt chunk of 4 sequences, every head, padded to a fixed number of rows
        dict(name="topk, 1000 rows, 128 heads", op="topk", seqs=4, rows=250, pad=24, H=128, K=2048, E=576, lo=1000,
             hi=16384, cache="bf16"),

        # one short sequence with a short system prompt: latency
        dict(name="shared, 1 query", op="shared", seqs=1, H=16, E=576, prefix=100, lo=0, hi=64, cache="bf16"),
        # a batch that answers questions on one long document
        dict(name="shared, 64 queries, 16 heads", op="shared", seqs=64, H=16, E=576, prefix=32768, lo=1, hi=512,
             cache="bf16"),
        # odd sizes, fp8 rows, contexts as long as the prefix
        dict(name="shared, 33 queries, 40 heads, fp8", op="shared", seqs=33, H=40, E=512, prefix=5001, lo=0, hi=5000,
             cache="fp8"),
        # every head of a large batch on a long document: bound by the matrix cores
        dict(name="shared, 64 queries, 128 heads", op="shared", seqs=64, H=128, E=576, prefix=32751, lo=1, hi=300,
             cache="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


MOST_FLOPS = 5.0e11


def draw(rng):
    op = rng.choice(["append", "topk", "shared"])
    E, cache = rng.choice([512, 576]), rng.choice(["bf16", "bf16", "fp8"])
    if op == "append":
        tokens = _log_uniform(rng, 1, 32768)
        return dict(op=op, tokens=tokens, seqs=rng.randint(1, min(tokens, 64)), E=E, input=rng.choice(["bf16", "f32"]),
                    cache=cache, index=rng.random() < 0.7, kv_pairs=rng.random() < 0.5,
                    index_pairs=rng.random() < 0.5)
    H = rng.choice([rng.randint(1, 128), 16, 32, 64, 128])
    per = 2.0 * H * (E + V)  # operations of one query and one key
    if op == "topk":
        K = _log_uniform(rng, 1, 2048)
        rows = rng.choice([1, 1, _log_uniform(rng, 1, 512)])
        seqs = _log_uniform(rng, 1, 128 if rows == 1 else 8)
        hi = _log_uniform(rng, 64, 32768)
        rows = max(1, min(rows, int(MOST_FLOPS / (per * K * seqs)), hi))
        return dict(op=op, seqs=seqs, rows=rows, pad=rng.choice([0, 0, rng.randint(1, 16)]), H=H, K=K, E=E,
                    lo=rng.choice([0, hi // 2, hi]), hi=hi, cache=cache)
    seqs = _log_uniform(rng, 1, 128)
    hi = _log_uniform(rng, 1, 4096)
    prefix = rng.choice([0] + [_log_uniform(rng, 64, 65536)] * 7)
    prefix = int(min(prefix, MOST_FLOPS / (per * seqs)))
    return dict(op=op, seqs=seqs, H=H, E=E, prefix=prefix, lo=rng.choice([0, hi]), hi=hi, cache=cache)


def _lens(case):
    """The sequences' lengths: part of the case, not of the seed."""
    r = random.Random("%d %d %d" % (case["seqs"], case["lo"], case["hi"]))
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]


def _split(total, parts):
    """`total` tokens over `parts` sequences, ragged: at least one each."""
    r = random.Random("%d %d" % (total, parts))
    cuts = sorted(r.sample(range(1, total), parts - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _row_bytes(case):
    return 2 * case["E"] if case["cache"] == "bf16" else case["E"] + 4


def work(case):
    E = case["E"]
    if case["op"] == "append":
        T, size = case["tokens"], 2 if case["input"] == "bf16" else 4
        width = E + (D if case["index"] else 0)
        longest = max(_split(T, case["seqs"]))
        nbytes = T * (width * size + 8 + _row_bytes(case) + (D + 4 if case["index"] else 0)) + longest * ROPE * 4
        return {"bytes": nbytes, "flops": 6 * (ROPE // 2) * T * (2 if case["index"] else 1)}
    H = case["H"]
    lens = _lens(case)
    if case["op"] == "topk":
        n = sum(min(case["K"], p) for c in lens for p in range(max(0, c - case["rows"]) + 1, c + 1))
        T = case["seqs"] * case["rows"] + case["pad"]
        rows = min(n, sum(lens))
        index = T * case["K"] * 4
    else:
        n = case["seqs"] * case["prefix"] + sum(lens)
        T = case["seqs"]
        rows = case["prefix"] + sum(lens)
        index = T * 4
    return {"bytes": rows * _row_bytes(case) + T * H * (E * 2 + V * 2 + 4) + index, "flops": 2 * n * H * (E + V)}


def _pool(case, pages, g, dev):
    """A latent pool with something in every slot, and the scales of fp8 rows."""
    E = case["E"]
    x = torch.randn((pages, PAGE, E), generator=g, device=dev, dtype=torch.bfloat16)
    if case["cache"] == "bf16":
        return x, None
    codes = torch.empty((pages, PAGE, E), device=dev, dtype=torch.uint8)
    codes.view(torch.float8_e4m3fn).copy_((x * 100).clamp_(-E4M3_MAX, E4M3_MAX))
    return codes, 0.005 + 0.01 * torch.rand((pages, PAGE), generator=g, device=dev)


def _table(lens, pages, g, dev, first=0):
    """Block table of sequences of `lens` tokens over the pages from `first` on, scattered."""
    need = [-(-n // PAGE) for n in lens]
    perm = (torch.randperm(pages - first, generator=g, device=dev) + first).to(torch.int32)
    width = max(1, max(need))
    table = torch.zeros((len(lens), width), dtype=torch.int32, device=dev)
    owned = torch.arange(width, device=dev)[None, :] < torch.tensor(need, device=dev)[:, None]
    table[owned] = perm[: sum(need)]
    return table


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    E = case["E"]
    if case["op"] == "append":
        T = case["tokens"]
        counts = _split(T, case["seqs"])
        before = random.Random(T).randint(0, 300)  # tokens of every sequence that are in the cache already
        lens = [before + n for n in counts]
        pages = sum(-(-n // PAGE) for n in lens) + 3
        cache, scale = _pool(case, pages, g, dev)
        far = max(lens)
        angle = torch.arange(far, device=dev, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, ROPE, 2, device=dev, dtype=torch.float64) / ROPE)
        seq = torch.repeat_interleave(torch.arange(len(counts), device=dev, dtype=torch.int32),
                                      torch.tensor(counts, device=dev))
        pos = torch.cat([torch.arange(before, n, device=dev, dtype=torch.int32) for n in lens])
        dt = DTYPES[case["input"]]
        st = dict(case=case, cache=cache, scale=scale, seq=seq, pos=pos, table=_table(lens, pages, g, dev),
                  cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(),
                  kv=torch.randn((T, E), generator=g, device=dev, dtype=dt), index_k=None, k_cache=None, k_scale=None)
        if case["index"]:
            st["index_k"] = torch.randn((T, D), generator=g, device=dev, dtype=dt)
            st["k_cache"] = torch.randint(0, 120, (pages, PAGE, D), generator=g, device=dev, dtype=torch.uint8)
            st["k_scale"] = 0.005 + 0.01 * torch.rand((pages, PAGE), generator=g, device=dev)
        return st
    H, B = case["H"], case["seqs"]
    lens = _lens(case)
    own_pages = sum(-(-n // PAGE) for n in lens)
    if case["op"] == "topk":
        R, K = case["rows"], case["K"]
        T = B * R + case["pad"]
        pages = own_pages + 1
        cache, scale = _pool(case, pages, g, dev)
        ctx = torch.tensor(lens, device=dev, dtype=torch.int64)
        n = (ctx[:, None] - R + 1 + torch.arange(R, device=dev)).clamp_(min=0).reshape(-1)  # positions a row sees
        n = torch.cat([n, torch.zeros(case["pad"], device=dev, dtype=torch.int64)])[:, None]
        j = torch.arange(K, device=dev)[None, :]
        lo, hi = j * n // K, (j + 1) * n // K  # K or fewer positions: all of them; more: one of each stratum
        u = torch.rand((T, K), generator=g, device=dev, dtype=torch.float64)
        idx = torch.where(n > K, lo + (u * (hi - lo)).long(), torch.where(j < n, j, -1)).to(torch.int32)
        seq = None
        if R > 1 or case["pad"]:
            seq = torch.cat([torch.arange(B, device=dev, dtype=torch.int32).repeat_interleave(R),
                             torch.full((case["pad"],), -1, device=dev, dtype=torch.int32)])
        return dict(case=case, cache=cache, scale=scale, table=_table(lens, pages, g, dev), idx=idx, seq=seq,
                    q=1.5 * torch.randn((T, H, E), generator=g, device=dev, dtype=torch.bfloat16))
    shared = -(-case["prefix"] // PAGE)
    pages = shared + own_pages + 1
    cache, scale = _pool(case, pages, g, dev)
    return dict(case=case, cache=cache, scale=scale, table=_table(lens, pages, g, dev, shared),
                prefix_table=torch.randperm(max(1, shared), generator=g, device=dev).to(torch.int32),
                lens=torch.tensor(lens, device=dev, dtype=torch.int32),
                q=1.5 * torch.randn((B, H, E), generator=g, device=dev, dtype=torch.bfloat16))


def _package():
    global _dsa
    if _dsa is None:
        import dsa_lightning_indexer_03_amd
        _dsa = dsa_lightning_indexer_03_amd
    return _dsa


def _softmax_scale(E):
    return 1.0 / math.sqrt(E)


def run(st):
    case = st["case"]
    return {"append": _append, "topk": _topk, "shared": _shared}[case["op"]](case, st)


# ---- the caches' write path -------------------------------------------------------------------------------------

def _rotated(x, cos, sin, first, pairs):
    """fp32 rows with the columns first .. first + ROPE rotated: pairs (2i, 2i+1), or halves (i, i + ROPE/2)."""
    y = x.float().clone()
    r = y[:, first:first + ROPE]
    a, b = (r[:, 0::2].clone(), r[:, 1::2].clone()) if pairs else (r[:, :ROPE // 2].clone(), r[:, ROPE // 2:].clone())
    u, w = a * cos - b * sin, b * cos + a * sin
    y[:, first:first + ROPE] = torch.stack([u, w], 2).flatten(1) if pairs else torch.cat([u, w], 1)
    return y


def _quantised(y):
    amax = y.abs().amax(1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
    return (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _append(case, st):
    if own:
        _package().cache_append_rope(st["kv"], st["seq"], st["pos"], st["table"], st["cache"], st["cos_sin"],
                                     latent_scale=st["scale"], kv_interleaved=case["kv_pairs"], index_k=st["index_k"],
                                     k_cache=st["k_cache"], k_scale=st["k_scale"],
                                     index_interleaved=case["index_pairs"])
    else:
        pos = st["pos"].long()
        slot = st["table"][st["seq"].long(), pos // PAGE].long() * PAGE + pos % PAGE
        cos, sin = st["cos_sin"][pos].split(ROPE // 2, 1)
        y = _rotated(st["kv"], cos, sin, case["E"] - ROPE, case["kv_pairs"])
        if case["cache"] == "bf16":
            st["cache"].view(-1, case["E"])[slot] = y.bfloat16()
        else:
            codes, scale = _quantised(y)
            st["cache"].view(-1, case["E"])[slot] = codes.view(torch.uint8)
            st["scale"].view(-1)[slot] = scale
        if case["index"]:
            codes, scale = _quantised(_rotated(st["index_k"], cos, sin, 0, case["index_pairs"]))
            st["k_cache"].view(-1, D)[slot] = codes.view(torch.uint8)
            st["k_scale"].view(-1)[slot] = scale
    out = {"latent": st["cache"] if case["cache"] == "bf16" else st["cache"].view(torch.float8_e4m3fn)}
    if case["cache"] == "fp8":
        out["latent_scale"] = st["scale"]
    if case["index"]:
        out["key"], out["key_scale"] = st["k_cache"].view(torch.float8_e4m3fn), st["k_scale"]
    return out


# ---- attention over the latent cache -----------------------------------------------------------------------------

def _rows(st, slots):
    """fp32 latent rows at these slots of the pool."""
    E = st["case"]["E"]
    if st["scale"] is None:
        return st["cache"].view(-1, E)[slots].float()
    return st["cache"].view(-1, E)[slots].view(torch.float8_e4m3fn).float() * st["scale"].view(-1)[slots][..., None]


def _softmax(s):
    """exp(s - max), its sum and the log of the sum of exp(s): rows without a finite score give zeros and -inf."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    return p, total, (m + total.log()).squeeze(-1)


def _topk(case, st):
    E = case["E"]
    if own:
        out, lse = _package().latent_attention_topk(st["q"], st["cache"], st["table"], st["idx"], V, _softmax_scale(E),
                                                    latent_scale=st["scale"], seq_ids=st["seq"], want_lse=True)
        return {"out": out, "lse": lse}
    idx = st["idx"].long()
    table = st["table"].long()
    valid = (idx >= 0) & (idx < table.shape[1] * PAGE)
    at = idx.clamp(min=0)
    if st["seq"] is None:
        page = torch.gather(table, 1, at // PAGE)
    else:
        valid &= (st["seq"] >= 0)[:, None]
        page = table[st["seq"].clamp(min=0).long()[:, None], at // PAGE]
    rows = _rows(st, page * PAGE + at % PAGE)
    s = torch.matmul(st["q"].float(), rows.transpose(1, 2)) * _softmax_scale(E)
    s = torch.where(valid[:, None, :], s, -math.inf)
    p, total, lse = _softmax(s)
    out = torch.matmul(p, rows[:, :, :V])
    return {"out": torch.where(total > 0, out / total, 0.0).bfloat16(), "lse": lse}


def _shared(case, st):
    E, L = case["E"], case["prefix"]
    if own:
        out, lse = _package().latent_attention_shared(st["q"], st["cache"], st["prefix_table"], L, st["table"],
                                                      st["lens"], V, _softmax_scale(E), latent_scale=st["scale"],
                                                      want_lse=True)
        return {"out": out, "lse": lse}
    B, H = case["seqs"], case["H"]
    q = st["q"].float()
    j = torch.arange(L, device=q.device)
    pre = _rows(st, st["prefix_table"].long()[j // PAGE] * PAGE + j % PAGE)
    j = torch.arange(st["table"].shape[1] * PAGE, device=q.device)
    rows = _rows(st, st["table"].long()[:, j // PAGE] * PAGE + j % PAGE)
    s_pre = torch.matmul(q.view(B * H, E), pre.t()).view(B, H, L)
    s_own = torch.matmul(q, rows.transpose(1, 2))
    s_own = torch.where((j[None, :] < st["lens"][:, None])[:, None, :], s_own, -math.inf)
    p, total, lse = _softmax(torch.cat([s_pre, s_own], 2) * _softmax_scale(E))
    out = torch.matmul(p[:, :, :L].reshape(B * H, L), pre[:, :V]).view(B, H, V) + \
        torch.matmul(p[:, :, L:], rows[:, :, :V])
    return {"out": torch.where(total > 0, out / total, 0.0).bfloat16(), "lse": lse}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def _exact_turn(x, pos, first, pairs):
    """Columns first .. first + ROPE as complex numbers, turned by the position's angle (the table's fp32 entries)."""
    y = x.double()
    r = y[:, first:first + ROPE]
    z = torch.complex(r[:, 0::2], r[:, 1::2]) if pairs else torch.complex(r[:, :ROPE // 2], r[:, ROPE // 2:])
    z = z * pos
    y[:, first:first + ROPE] = torch.view_as_real(z).flatten(1) if pairs else torch.cat([z.real, z.imag], 1)
    return y


def _exact_append(case, st):
    turn = st["cos_sin"].double()[st["pos"].long()]
    turn = torch.complex(turn[:, :ROPE // 2], turn[:, ROPE // 2:])
    pos = st["pos"].tolist()
    table = st["table"].cpu().tolist()
    slot = torch.tensor([table[b][p // PAGE] * PAGE + p % PAGE for b, p in zip(st["seq"].tolist(), pos)],
                        device=turn.device)
    out = {}
    for name, x, cache, scale, first, pairs in (
            ("latent", st["kv"], st["cache"], st["scale"], case["E"] - ROPE, case["kv_pairs"]),
            ("key", st["index_k"], st["k_cache"], st["k_scale"], 0, case["index_pairs"])):
        if x is None:
            continue
        y = _exact_turn(x, turn, first, pairs)
        if cache.dtype == torch.bfloat16:
            kept = cache.double()
        else:
            kept = cache.view(torch.float8_e4m3fn).double()
            by = y.abs().amax(1) / 448
            y = y / by[:, None]
            out[name + "_scale"] = scale.double().view(-1).index_put((slot,), by).view(scale.shape)
        out[name] = kept.view(-1, y.shape[1]).index_put((slot,), y).view(kept.shape)
    return out


def _exact_attend(q, rows, scale):
    """One block of queries [.., h, E] over the keys [.., n, E] in 64 bits."""
    if rows.shape[-2] == 0:
        return q.new_zeros(q.shape[:-1] + (V,)), q.new_full(q.shape[:-1], -math.inf)
    s = q @ rows.transpose(-1, -2) * scale
    lse = torch.logsumexp(s, -1)
    return torch.exp(s - lse[..., None]) @ rows[..., :V], lse


def _exact_rows(st, slots):
    x = st["cache"].view(-1, st["case"]["E"])[slots]
    if st["scale"] is None:
        return x.double()
    return x.view(torch.float8_e4m3fn).double() * st["scale"].double().view(-1)[slots][:, None]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, st)
    scale = 1.0 / math.sqrt(case["E"])
    outs, lses = [], []
    if case["op"] == "topk":
        for t in range(st["q"].shape[0]):
            b = t if st["seq"] is None else t // case["rows"] if t < case["seqs"] * case["rows"] else -1
            at = st["idx"][t].long()
            at = at[at >= 0] if b >= 0 else at[:0]
            slots = st["table"][b].long()[at // PAGE] * PAGE + at % PAGE
            o, l = _exact_attend(st["q"][t].double(), _exact_rows(st, slots), scale)
            outs.append(o)
            lses.append(l)
        return {"out": torch.stack(outs), "lse": torch.stack(lses)}
    j = torch.arange(case["prefix"], device=st["q"].device)
    pre = _exact_rows(st, st["prefix_table"].long()[j // PAGE] * PAGE + j % PAGE)
    for b, n in enumerate(_lens(case)):
        j = torch.arange(n, device=st["q"].device)
        mine = _exact_rows(st, st["table"][b].long()[j // PAGE] * PAGE + j % PAGE)
        o, l = _exact_attend(st["q"][b].double(), torch.cat([pre, mine]), scale)
        outs.append(o)
        lses.append(l)
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
