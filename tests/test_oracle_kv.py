"""Pins of the oracle for attention with grouped keys and values: closed forms,
loops written out, and torch's own operations on the CPU."""
import math

import numpy as np
import torch

from oracle.kv import attend, decode, grouped, place, positions, prompt


def test_closed_forms():
    v = np.array([[1.0, 2.0], [5.0, -4.0]])
    out, lse, _, _ = attend(np.zeros((1, 3)), np.ones((2, 3)), v, 0.7)         # equal scores: the mean
    assert np.allclose(out, [[3.0, -1.0]]) and np.isclose(lse[0], math.log(2))
    q, k = np.array([[1.0, 0.0]]), np.array([[math.log(3.0), 9.0], [0.0, 7.0]])
    out, lse, _, _ = attend(q, k, v, 1.0)                                      # weights 3 : 1
    assert np.allclose(out, [[2.0, 0.5]]) and np.isclose(lse[0], math.log(4))
    out, lse, eo, el = attend(q, k[:0], v[:0], 1.0)
    assert not out.any() and lse[0] == -np.inf and not eo.any() and not el.any()


def test_heads_read_their_group():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(6, 4)), rng.normal(size=(5, 3, 4)), rng.normal(size=(5, 3, 2))
    out, lse, _, _ = grouped(q, k, v, 0.5)
    for h in range(6):
        s = [0.5 * sum(q[h, d] * k[j, h // 2, d] for d in range(4)) for j in range(5)]
        w = [math.exp(x) for x in s]
        assert np.isclose(lse[h], math.log(sum(w)))
        for c in range(2):
            assert np.isclose(out[h, c], sum(w[j] * v[j, h // 2, c] for j in range(5)) / sum(w))


def test_prompt_is_causal_and_packed():
    rng = np.random.default_rng(1)
    cu, T = [0, 3, 3, 8], 10
    q, k, v = rng.normal(size=(T, 2, 4)), rng.normal(size=(T, 1, 4)), rng.normal(size=(T, 1, 3))
    out, lse, _, _ = prompt(q, k, v, cu, 1.0)
    for a, b in zip(cu, cu[1:]):
        if b > a:
            s = torch.einsum("ihd,jd->hij", torch.from_numpy(q[a:b]), torch.from_numpy(k[a:b, 0]))
            s = s.masked_fill(torch.ones(b - a, b - a, dtype=torch.bool).triu(1), -math.inf)
            assert np.allclose(lse[a:b], torch.logsumexp(s, 2).t().numpy())
            assert np.allclose(out[a:b], (s.softmax(2) @ torch.from_numpy(v[a:b, 0])).transpose(0, 1).numpy())
    assert not out[8:].any() and np.isneginf(lse[8:]).all()


def test_positions_and_places():
    assert positions([3, -1, 7, 0, 5, 3], 6).tolist() == [3, 0, 5, 3]
    page, slot = place([0, 63, 64, 130], [4, 9, -2], 9)
    assert page.tolist() == [4, 4, -1, -1] and slot.tolist() == [0, 63, 0, 2]


def test_decode_reads_through_the_table():
    rng = np.random.default_rng(2)
    k, v = rng.normal(size=(4, 2, 64, 3)), rng.normal(size=(4, 2, 64, 3))
    q, table = rng.normal(size=(2, 4, 3)), np.array([[2, 0], [1, 3]])
    rows = lambda x, b: np.concatenate([x[p].transpose(1, 0, 2) for p in table[b]])   # noqa: E731
    got = decode(q, k, v, table, [70, 5], 0.3)
    for b, n in enumerate([70, 5]):
        want = grouped(q[b], rows(k, b)[:n], rows(v, b)[:n], 0.3)
        assert np.allclose(got[b][0], want[0]) and np.allclose(got[b][1], want[1])
    got = decode(q, k, v, table, [70, 5], 0.3, idx=[[69, 69, 1, -1], [5, 6, -1, 70]])
    want = grouped(q[0], rows(k, 0)[[69, 69, 1]], rows(v, 0)[[69, 69, 1]], 0.3)
    assert np.allclose(got[0][0], want[0]) and np.isneginf(got[1][1]).all()


def test_bounds_hold_for_the_computation_they_describe():
    """fp32 scores and sums, bf16 probabilities and results, by torch on the CPU."""
    rng = np.random.default_rng(3)
    for n, D, V in ((1, 64, 64), (70, 128, 128), (300, 192, 128)):
        q, k, v = (torch.from_numpy(rng.normal(size=s)).bfloat16() for s in ((5, D), (n, D), (n, V)))
        s = (1.5 * q.float()) @ k.float().t() * D ** -0.5
        m = s.amax(1, keepdim=True)
        p = torch.exp(s - m)
        total = p.sum(1, keepdim=True)
        out = ((p.bfloat16().float() @ v.float()) / total).bfloat16().double().numpy()
        lse = (m + total.log())[:, 0].double().numpy()
        o, l, eo, el = attend(1.5 * q.double().numpy(), k.double().numpy(), v.double().numpy(), D ** -0.5)
        assert (np.abs(out - o) <= eo).all() and (np.abs(lse - l) <= el).all()
        assert (eo <= 0.05 * (np.abs(o) + 1)).all()
