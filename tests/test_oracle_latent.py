"""Pins of oracle/latent.py: closed forms and properties that do not share its
formulas."""
import numpy as np

from oracle.latent import attend, rotate, slots


def test_rotation_is_a_complex_product():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(5, 40))
    ang = rng.uniform(-9, 9, size=(5, 8))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    for first, pairs in ((0, True), (24, True), (0, False), (24, False), (7, False)):
        y, err = rotate(x, cs, first, pairs)
        r = x[:, first:first + 16]
        z = r[:, 0::2] + 1j * r[:, 1::2] if pairs else r[:, :8] + 1j * r[:, 8:]
        z = z * np.exp(1j * ang)
        w = np.empty_like(r)
        if pairs:
            w[:, 0::2], w[:, 1::2] = z.real, z.imag
        else:
            w[:, :8], w[:, 8:] = z.real, z.imag
        assert np.allclose(y[:, first:first + 16], w, rtol=0, atol=1e-12)
        keep = np.ones(40, bool)
        keep[first:first + 16] = False
        assert np.array_equal(y[:, keep], x[:, keep]) and not err[:, keep].any()
        assert np.allclose((y ** 2).sum(1), (x ** 2).sum(1))


def test_rotation_depends_on_the_difference_of_positions():
    rng = np.random.default_rng(2)
    a, b = rng.normal(size=(2, 1, 16))
    freq = 10000.0 ** (-np.arange(0, 16, 2) / 16)

    def at(x, p):
        return rotate(x, np.concatenate([np.cos(p * freq), np.sin(p * freq)])[None], 0, True)[0]

    assert np.isclose((at(a, 70) * at(b, 3)).sum(), (at(a, 1067) * at(b, 1000)).sum())


def test_slots_name_only_what_exists():
    table = np.array([[3, 0], [9, -1]], dtype=np.int32)
    s = slots([0, 0, 0, 1, 1, 2, -1, 0, 0], [0, 65, 128, 0, 64, 0, 0, -1, 70], table, 9, limit=70)
    assert s.tolist() == [192, 1, -1, -1, -1, -1, -1, -1, -1]


def test_attention_closed_forms():
    rng = np.random.default_rng(3)
    rows = rng.normal(size=(6, 8))
    q = np.zeros((2, 8))
    out, lse, err, _ = attend(q, rows, 1.0, 5)       # no preference: the mean
    assert np.allclose(out, rows[:, :5].mean(0)) and np.allclose(lse, np.log(6)) and (err > 0).all()
    q = rng.normal(size=(2, 8))
    one, lse1, _, _ = attend(q, rows[:1], 0.5, 5)    # one row: that row
    assert np.allclose(one, rows[0, :5]) and np.allclose(lse1, 0.5 * q @ rows[0])
    twice, lse2, _, _ = attend(q, np.concatenate([rows, rows]), 0.5, 5)   # every row twice: the same mean
    once, lse3, _, _ = attend(q, rows, 0.5, 5)
    assert np.allclose(twice, once) and np.allclose(lse2, lse3 + np.log(2))
    none, lse0, _, _ = attend(q, rows[:0], 0.5, 5)
    assert not none.any() and np.isneginf(lse0).all()


def test_parts_join_by_their_lse():
    rng = np.random.default_rng(4)
    q, rows = rng.normal(size=(3, 8)), rng.normal(size=(11, 8))
    o, l, _, _ = attend(q, rows, 0.7, 8)
    o1, l1, _, _ = attend(q, rows[:4], 0.7, 8)
    o2, l2, _, _ = attend(q, rows[4:], 0.7, 8)
    w = np.exp(l1 - np.logaddexp(l1, l2))[:, None]
    assert np.allclose(o, w * o1 + (1 - w) * o2) and np.allclose(l, np.logaddexp(l1, l2))
