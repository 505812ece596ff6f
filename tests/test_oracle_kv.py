"""Pins of oracle/kv.py: closed forms and identities, on the CPU."""
import numpy as np

from oracle import kv as okv


def test_rope_turns_and_keeps_lengths():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 16))
    pos, f = np.array([0, 1, -3, 100, 7]), 10.0 ** -np.arange(4)
    for layout in ("half", "interleaved"):
        y = okv.rope(x, pos, f, layout)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 8:], x[..., 8:])
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        back = okv.rope(y, -pos, f, layout)
        assert np.allclose(back, x)
        assert np.allclose(okv.rope(x, pos, f, layout, 2.0)[..., :8], 2 * y[..., :8])
    quarter = okv.rope(np.array([[[1.0, 2.0, 3.0, 4.0]]]), [1], [np.pi / 2, np.pi], "interleaved")
    assert np.allclose(quarter, [[[-2.0, 1.0, -3.0, -4.0]]])
    quarter = okv.rope(np.array([[[1.0, 2.0, 3.0, 4.0]]]), [1], [np.pi / 2, np.pi], "half")
    assert np.allclose(quarter, [[[-3.0, -2.0, 1.0, -4.0]]])


def test_products_depend_on_distance_alone():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 16))
    f = 100.0 ** (-np.arange(8) / 8)
    dots = [float((okv.rope(q, [p + 5], f) * okv.rope(k, [p], f)).sum()) for p in (0, 3, 1000)]
    assert np.allclose(dots, dots[0])


def test_slots():
    s, p = okv.slots([0, 2, 2, 3], [18, 5, 1], [[7, 3], [1, 1], [2, 0]], 16, 4)
    assert s.tolist() == [3 * 16, 3 * 16 + 1, 2 * 16, -1] and p.tolist() == [16, 17, 0, 0]


def test_attend_closed_forms():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 6, 1, 4))
    q = rng.standard_normal((3, 2, 4))
    out, lse, mag, _ = okv.attend(q, k, v, okv.visible(3, 6), 0.0)      # a scale of zero: means of what is in sight
    for i in range(3):
        assert np.allclose(out[i, 0], v[: 4 + i, 0].mean(0)) and np.isclose(lse[i, 1], np.log(4 + i))
        assert np.allclose(mag[i, 0], np.abs(v[: 4 + i, 0]).mean(0))
    out, lse, _, _ = okv.attend(q, k, v, okv.visible(3, 6, window=1), 0.7)  # a window of one: the token itself
    assert np.allclose(out[:, 0], v[3:, 0]) and np.allclose(lse[2, 0], 0.7 * k[5, 0] @ q[2, 0])
    out, lse, _, _ = okv.attend(q, k, v, np.zeros((3, 6), bool), 0.7)
    assert (out == 0).all() and np.isneginf(lse).all()
    assert okv.visible(2, 4, causal=False).all() and okv.visible(2, 4, causal=False, window=2).tolist() == [
        [False, True, True, True], [False, False, True, True]]
