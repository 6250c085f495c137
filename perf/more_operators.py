"""Cases for the attention of layers that keep keys and values of their own for groups of heads: the write of both
paged caches with the position rotation, causal attention over whole prompts, and attention of one new token per
sequence over the caches, at every position or at the indexer's selection.

The caches hold, for each of G key/value heads, a D-wide key row and a D-wide value row per token, in pages of 64
tokens: [pages][G][64][D], bf16, or e4m3 codes with one fp32 scale per row. Query head h reads head h // (H / G)."""
import math
import random

import torch

_dsa = None  # the package, imported on the first call that needs it
own = False

PAGE = 64
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one new token of one sequence: a decode step's write, launch latency alone
        dict(name="append, 1 token", op="append", tokens=1, seqs=1, G=8, D=128, R=128, pairs=False, input="bf16",
             cache="bf16"),
        # a prompt chunk over ragged sequences, fp32 projections, half of each key rotated, fp8 rows, narrow heads
        dict(name="append, 4099 tokens, f32 to fp8", op="append", tokens=4099, seqs=7, G=4, D=64, R=32, pairs=True,
             input="f32", cache="fp8"),
        # the largest prompt the indexer's headline workload prefills
        dict(name="append, 32768 tokens", op="append", tokens=32768, seqs=3, G=8, D=128, R=128, pairs=False,
             input="bf16", cache="bf16"),

        # one short prompt, a key/value head for each query head, keys with a rotary part of their own: latency
        dict(name="prompt, 61 tokens", op="prompt", tokens=61, seqs=1, pad=0, H=16, G=16, D=192, V=128),
        # a batch of prompts too short for a selection, padded to a fixed number of rows
        dict(name="prompt, 16 sequences, 16 heads of 192", op="prompt", tokens=12007, seqs=16, pad=281, H=16, G=16,
             D=192, V=128),
        # ragged prompts, narrow heads, many query heads to one key/value head
        dict(name="prompt, 5 sequences, 28 heads over 4", op="prompt", tokens=9001, seqs=5, pad=0, H=28, G=4, D=64,
             V=64),
        # one long document, grouped heads: bound by the matrix cores
        dict(name="prompt, 32768 tokens, 16 heads over 2", op="prompt", tokens=32768, seqs=1, pad=0, H=16, G=2, D=128,
             V=128),

        # one short sequence: latency
        dict(name="decode, 1 sequence of 100", op="decode", seqs=1, H=32, G=8, D=128, lo=100, hi=100, K=0,
             cache="bf16"),
        # one sequence at the longest context: the work of 8 key/value heads has to fill the card
        dict(name="decode, 1 sequence of 131072, fp8", op="decode", seqs=1, H=64, G=8, D=128, lo=131072, hi=131072,
             K=0, cache="fp8"),
        # a serving batch's decode step: bound by the cache's bytes
        dict(name="decode, 64 sequences", op="decode", seqs=64, H=32, G=8, D=128, lo=4096, hi=32768, K=0,
             cache="bf16"),
        # odd batch and group of heads, narrow heads, short contexts, an empty one among them
        dict(name="decode, 37 sequences, 21 heads over 3, fp8", op="decode", seqs=37, H=21, G=3, D=64, lo=0, hi=6000,
             K=0, cache="fp8"),
        # a serving batch at the indexer's selection of 2048 positions each
        dict(name="decode, 64 sequences, 2048 selected", op="decode", seqs=64, H=32, G=8, D=128, lo=1000, hi=32768,
             K=2048, cache="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


MOST_FLOPS = 3.0e12   # a prompt
MOST_ROWS = 2.0e9     # bytes of the rows that a decode step reads


def draw(rng):
    op = rng.choice(["append", "prompt", "decode"])
    G = rng.choice([1, 2, 3, 4, 8, 16])
    if op == "append":
        tokens = _log_uniform(rng, 1, 32768)
        D = rng.choice([64, 128])
        G = min(G, 8)
        return dict(op=op, tokens=tokens, seqs=rng.randint(1, min(tokens, 64)), G=G, D=D,
                    R=rng.choice([0, 16, D // 2, D]), pairs=rng.random() < 0.5, input=rng.choice(["bf16", "f32"]),
                    cache=rng.choice(["bf16", "fp8"]))
    H = G * rng.choice([1, 2, 4, 5, 7, 8, 16])
    H = H if H <= 64 else G * 2
    if op == "prompt":
        D, V = rng.choice([(64, 64), (128, 128), (192, 128)])
        tokens = _log_uniform(rng, 1, 32768)
        case = dict(op=op, tokens=tokens, seqs=min(tokens, _log_uniform(rng, 1, 32)),
                    pad=rng.choice([0, 0, rng.randint(1, 300)]), H=H, G=G, D=D, V=V)
        while work(case)["flops"] > MOST_FLOPS:
            case["tokens"] = max(1, int(0.8 * case["tokens"]))
            case["seqs"] = min(case["seqs"], case["tokens"])
        return case
    case = dict(op=op, seqs=_log_uniform(rng, 1, 128), H=H, G=G, D=rng.choice([64, 128]), lo=0,
                hi=_log_uniform(rng, 1, 131072), K=rng.choice([0, 0, _log_uniform(rng, 1, 2048)]),
                cache=rng.choice(["bf16", "bf16", "fp8"]))
    most = int(MOST_ROWS / (case["seqs"] * G * 2 * _row_bytes(case)))
    case["hi"] = max(1, min(case["hi"], most))
    case["lo"] = rng.choice([0, case["hi"] // 2, case["hi"]])
    return case


def _lens(case):
    """The contexts' lengths: part of the case, not of the seed."""
    r = random.Random("%d %d %d" % (case["seqs"], case["lo"], case["hi"]))
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]


def _split(total, parts):
    """`total` tokens over `parts` sequences, ragged: at least one each."""
    r = random.Random("%d %d" % (total, parts))
    cuts = sorted(r.sample(range(1, total), parts - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _row_bytes(case):
    return 2 * case["D"] if case["cache"] == "bf16" else case["D"] + 4


def work(case):
    G, D = case["G"], case["D"]
    if case["op"] == "append":
        T, size = case["tokens"], DTYPES[case["input"]].itemsize
        longest = max(_split(T, case["seqs"]))
        return {"bytes": T * (2 * G * (D * size + _row_bytes(case)) + 8) + longest * case["R"] * 4,
                "flops": 3 * case["R"] * G * T}
    H = case["H"]
    if case["op"] == "prompt":
        V, T = case["V"], case["tokens"] + case["pad"]
        pairs = sum(n * (n + 1) // 2 for n in _split(case["tokens"], case["seqs"]))
        return {"bytes": 2 * T * (H * (D + V) + G * (D + V)) + 4 * T * H, "flops": 2 * pairs * H * (D + V)}
    n = sum(min(case["K"], c) if case["K"] else c for c in _lens(case))
    nbytes = n * G * 2 * _row_bytes(case) + case["seqs"] * (H * (4 * D + 4) + 4 + 4 * case["K"])
    return {"bytes": nbytes, "flops": 4 * n * H * D}


def _pool(case, pages, g, dev):
    """A pool of key or value rows with something in every slot, and the scales of fp8 rows."""
    G, D = case["G"], case["D"]
    x = torch.randn((pages, G, PAGE, D), generator=g, device=dev, dtype=torch.bfloat16)
    if case["cache"] == "bf16":
        return x, None
    codes = torch.empty((pages, G, PAGE, D), device=dev, dtype=torch.uint8)
    codes.view(torch.float8_e4m3fn).copy_((x * 100).clamp_(-E4M3_MAX, E4M3_MAX))
    return codes, 0.005 + 0.01 * torch.rand((pages, G, PAGE), generator=g, device=dev)


def _table(lens, pages, g, dev):
    """Block table of sequences of `lens` tokens, their pages scattered over the pool."""
    need = [-(-n // PAGE) for n in lens]
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    width = max(1, max(need))
    table = torch.zeros((len(lens), width), dtype=torch.int32, device=dev)
    owned = torch.arange(width, device=dev)[None, :] < torch.tensor(need, device=dev)[:, None]
    table[owned] = perm[: sum(need)]
    return table


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    G, D = case["G"], case["D"]
    if case["op"] == "append":
        T = case["tokens"]
        counts = _split(T, case["seqs"])
        before = random.Random(T).randint(0, 300)  # tokens of every sequence that are in the cache already
        lens = [before + n for n in counts]
        pages = sum(-(-n // PAGE) for n in lens) + 3
        st = dict(case=case, table=_table(lens, pages, g, dev), cos_sin=None)
        for name in ("k", "v"):
            st[name + "_cache"], st[name + "_scale"] = _pool(case, pages, g, dev)
        if case["R"]:
            R = case["R"]
            angle = torch.arange(max(lens), device=dev, dtype=torch.float64)[:, None] * \
                10000.0 ** (-torch.arange(0, R, 2, device=dev, dtype=torch.float64) / R)
            st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        st["seq"] = torch.repeat_interleave(torch.arange(len(counts), device=dev, dtype=torch.int32),
                                            torch.tensor(counts, device=dev))
        st["pos"] = torch.cat([torch.arange(before, n, device=dev, dtype=torch.int32) for n in lens])
        # keys and values side by side, as one projection makes them
        both = torch.randn((T, 2, G, D), generator=g, device=dev, dtype=DTYPES[case["input"]])
        st["k"], st["v"] = both[:, 0], both[:, 1]
        return st
    H = case["H"]
    if case["op"] == "prompt":
        T, V = case["tokens"] + case["pad"], case["V"]
        counts = _split(case["tokens"], case["seqs"])
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
        return dict(case=case, cu_host=cu, cu=torch.tensor(cu, device=dev, dtype=torch.int32),
                    q=1.5 * torch.randn((T, H, D), generator=g, device=dev, dtype=torch.bfloat16),
                    k=torch.randn((T, G, D), generator=g, device=dev, dtype=torch.bfloat16),
                    v=torch.randn((T, G, V), generator=g, device=dev, dtype=torch.bfloat16))
    B, K = case["seqs"], case["K"]
    lens = _lens(case)
    pages = sum(-(-n // PAGE) for n in lens) + 1
    st = dict(case=case, table=_table(lens, pages, g, dev), longest=max(lens), idx=None,
              lens=torch.tensor(lens, device=dev, dtype=torch.int32),
              q=1.5 * torch.randn((B, H, D), generator=g, device=dev, dtype=torch.bfloat16))
    for name in ("k", "v"):
        st[name + "_cache"], st[name + "_scale"] = _pool(case, pages, g, dev)
    if K:
        n = torch.tensor(lens, device=dev, dtype=torch.int64)[:, None]
        j = torch.arange(K, device=dev)[None, :]
        lo, hi = j * n // K, (j + 1) * n // K  # K or fewer positions: all of them; more: one of each stratum
        u = torch.rand((B, K), generator=g, device=dev, dtype=torch.float64)
        st["idx"] = torch.where(n > K, lo + (u * (hi - lo)).long(), torch.where(j < n, j, -1)).to(torch.int32)
    return st


def _package():
    global _dsa
    if _dsa is None:
        import dsa_lightning_indexer_03_amd
        _dsa = dsa_lightning_indexer_03_amd
    return _dsa


def run(st):
    case = st["case"]
    return {"append": _append, "prompt": _prompt, "decode": _decode}[case["op"]](case, st)


# ---- the caches' write path -------------------------------------------------------------------------------------

def _rotated(x, cos, sin, pairs):
    """fp32 rows [T, G, D] with their first 2 * cos.shape[-1] columns rotated: pairs (2i, 2i+1), or halves."""
    y = x.float().clone()
    half = cos.shape[-1]
    r = y[..., :2 * half]
    a, b = (r[..., 0::2].clone(), r[..., 1::2].clone()) if pairs else (r[..., :half].clone(), r[..., half:].clone())
    u, w = a * cos - b * sin, b * cos + a * sin
    y[..., :2 * half] = torch.stack([u, w], 3).flatten(2) if pairs else torch.cat([u, w], 2)
    return y


def _quantised(y):
    amax = y.abs().amax(-1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
    return (y / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _append(case, st):
    if own:
        _package().kv_append_rope(st["k"], st["v"], st["seq"], st["pos"], st["table"], st["k_cache"], st["v_cache"],
                                  cos_sin=st["cos_sin"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                                  interleaved=case["pairs"])
    else:
        pos = st["pos"].long()
        page, slot = st["table"][st["seq"].long(), pos // PAGE].long(), pos % PAGE
        k = st["k"].float()
        if case["R"]:
            cos, sin = st["cos_sin"][pos][:, None].split(case["R"] // 2, 2)
            k = _rotated(k, cos, sin, case["pairs"])
        for name, y in (("k", k), ("v", st["v"].float())):
            if case["cache"] == "bf16":
                st[name + "_cache"][page, :, slot] = y.bfloat16()
            else:
                codes, scale = _quantised(y)
                st[name + "_cache"][page, :, slot] = codes.view(torch.uint8)
                st[name + "_scale"][page, :, slot] = scale
    if case["cache"] == "bf16":
        return {"key": st["k_cache"], "value": st["v_cache"]}
    return {"key": st["k_cache"].view(torch.float8_e4m3fn), "key_scale": st["k_scale"],
            "value": st["v_cache"].view(torch.float8_e4m3fn), "value_scale": st["v_scale"]}


# ---- attention ---------------------------------------------------------------------------------------------------

def _scale(case):
    return 1.0 / math.sqrt(case["D"])


def _softmax(s):
    """exp(s - max), its sum and the log of the sum of exp(s): rows without a finite score give zeros and -inf."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    return p, total, (m + total.log()).squeeze(-1)


SCORES = 1 << 28  # scores that the plain forms hold at once


def _prompt(case, st):
    if own:
        out, lse = _package().prompt_attention(st["q"], st["k"], st["v"], st["cu"], _scale(case), want_lse=True)
        return {"out": out, "lse": lse}
    H, G, V = case["H"], case["G"], case["V"]
    T, R = st["q"].shape[0], H // G
    out = torch.zeros((T, H, V), device=st["q"].device, dtype=torch.bfloat16)
    lse = torch.full((T, H), -math.inf, device=st["q"].device)
    cu = st["cu_host"]
    for a, b in zip(cu, cu[1:]):
        n = b - a
        step = max(1, min(n, SCORES // (n * R)))
        for h in range(G):
            k, v = st["k"][a:b, h].float(), st["v"][a:b, h].float()
            for i in range(0, n, step):
                e = min(n, i + step)
                q = st["q"][a + i:a + e, h * R:(h + 1) * R].float().reshape(-1, case["D"])
                s = torch.matmul(q, k[:e].t()).view(e - i, R, e) * _scale(case)
                seen = torch.arange(e, device=s.device)[None, :] <= torch.arange(i, e, device=s.device)[:, None]
                p, total, l = _softmax(torch.where(seen[:, None, :], s, -math.inf))
                o = torch.matmul(p.view(-1, e), v[:e]).view(e - i, R, V) / total
                out[a + i:a + e, h * R:(h + 1) * R] = o.bfloat16()
                lse[a + i:a + e, h * R:(h + 1) * R] = l
    return {"out": out, "lse": lse}


def _rows(st, name, page, slot):
    """fp32 rows [..., G, D] at these pages and slots."""
    x = st[name + "_cache"]
    if st[name + "_scale"] is None:
        return x[page, :, slot].float()
    return x[page, :, slot].view(torch.float8_e4m3fn).float() * st[name + "_scale"][page, :, slot][..., None]


def _decode(case, st):
    if own:
        out, lse = _package().kv_attention_decode(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"],
                                                  _scale(case), topk_idx=st["idx"], max_context_len=st["longest"],
                                                  k_scale=st["k_scale"], v_scale=st["v_scale"], want_lse=True)
        return {"out": out, "lse": lse}
    B, H, G, D = case["seqs"], case["H"], case["G"], case["D"]
    R = H // G
    outs, lses = [], []
    n = case["K"] or max(1, st["longest"])
    step = max(1, SCORES // (n * G * D))
    for i in range(0, B, step):
        e = min(B, i + step)
        at = st["idx"][i:e].long() if case["K"] else torch.arange(n, device=st["q"].device).expand(e - i, n)
        valid = (at >= 0) & (at < st["lens"][i:e, None])
        at = at.clamp(min=0)
        page, slot = torch.gather(st["table"][i:e].long(), 1, at // PAGE), at % PAGE
        k = _rows(st, "k", page, slot).permute(0, 2, 1, 3).reshape(-1, n, D)
        v = _rows(st, "v", page, slot).permute(0, 2, 1, 3).reshape(-1, n, D)
        q = st["q"][i:e].float().view(-1, R, D)
        s = torch.matmul(q, k.transpose(1, 2)).view(e - i, G, R, n) * _scale(case)
        p, total, l = _softmax(torch.where(valid[:, None, None, :], s, -math.inf))
        o = torch.matmul(p.view(-1, R, n), v).view(e - i, G, R, D)
        outs.append(torch.where(total > 0, o / total, 0.0).reshape(e - i, H, D).bfloat16())
        lses.append(l.reshape(e - i, H))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def _exact_append(case, st):
    pos = st["pos"].tolist()
    table = st["table"].cpu().tolist()
    dev = st["k"].device
    page = torch.tensor([table[b][p // PAGE] for b, p in zip(st["seq"].tolist(), pos)], device=dev)
    slot = torch.tensor([p % PAGE for p in pos], device=dev)
    out = {}
    for name, key in (("k", "key"), ("v", "value")):
        y = st[name].double()
        if name == "k" and case["R"]:
            # the rotated columns as complex numbers, turned by the position's angle (the table's fp32 entries)
            half = case["R"] // 2
            turn = st["cos_sin"].double()[st["pos"].long()][:, None]
            turn = torch.complex(turn[..., :half], turn[..., half:])
            r = y[..., :2 * half]
            z = torch.complex(r[..., 0::2], r[..., 1::2]) if case["pairs"] else \
                torch.complex(r[..., :half], r[..., half:])
            z = z * turn
            z = torch.view_as_real(z).flatten(2) if case["pairs"] else torch.cat([z.real, z.imag], 2)
            y = torch.cat([z, y[..., 2 * half:]], 2)
        cache, scale = st[name + "_cache"], st[name + "_scale"]
        if scale is None:
            kept = cache.double()
        else:
            kept = cache.view(torch.float8_e4m3fn).double()
            by = y.abs().amax(2) / 448
            y = y / by[..., None]
            kept_scale = scale.double()
            kept_scale[page, :, slot] = by
            out[key + "_scale"] = kept_scale
        kept[page, :, slot] = y
        out[key] = kept
    return out


def _exact_head(q, k, v, scale, seen=None):
    """Rows q [m, D] over keys k [n, D] in 64 bits; `seen` [m, n]: what each row sees (None: all)."""
    s = q @ k.t() * scale
    if seen is not None:
        s = s.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, 1)
    return torch.exp(s - lse[:, None]) @ v, lse


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, st)
    H, R = case["H"], case["H"] // case["G"]
    scale = 1.0 / math.sqrt(case["D"])
    q = st["q"].double()
    out = torch.zeros(q.shape[:2] + st["v" if case["op"] == "prompt" else "v_cache"].shape[-1:], device=q.device,
                      dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, device=q.device, dtype=torch.float64)
    if case["op"] == "prompt":
        for a, b in zip(st["cu_host"], st["cu_host"][1:]):
            for h in range(H):
                k, v = st["k"][a:b, h // R].double(), st["v"][a:b, h // R].double()
                for i in range(a, b, 4096):
                    e = min(b, i + 4096)
                    seen = torch.ones((e - i, e - a), dtype=torch.bool, device=q.device).tril(i - a)
                    out[i:e, h], lse[i:e, h] = _exact_head(q[i:e, h], k[:e - a], v[:e - a], scale, seen)
        return {"out": out, "lse": lse}
    for b, n in enumerate(_lens(case)):
        at = torch.arange(n, device=q.device)
        if case["K"]:
            at = st["idx"][b].long()
            at = at[at >= 0]
        if at.numel() == 0:
            continue
        page, slot = st["table"][b].long()[at // PAGE], at % PAGE
        for h in range(H):
            rows = []
            for name in ("k", "v"):
                x = st[name + "_cache"][page, h // R, slot]
                if st[name + "_scale"] is None:
                    rows.append(x.double())
                else:
                    rows.append(x.view(torch.float8_e4m3fn).double() *
                                st[name + "_scale"].double()[page, h // R, slot][:, None])
            out[b, h:h + 1], lse[b, h:h + 1] = _exact_head(q[b, h:h + 1], rows[0], rows[1], scale)
    return {"out": out, "lse": lse}
