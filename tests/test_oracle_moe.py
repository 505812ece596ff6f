"""CPU pins of the mixture-of-experts oracle: hand-worked rows and closed forms."""
import numpy as np
import pytest

from oracle import moe


def test_route_softmax_by_hand():
    x = np.log(np.array([[1.0, 4.0, 2.0, 1.0]]))            # softmax 1/8, 1/2, 1/4, 1/8
    ids, w = moe.route(x, 2, renormalize=False)
    assert ids.tolist() == [[1, 2]] and np.allclose(w, [[0.5, 0.25]], rtol=1e-15)
    ids, w = moe.route(x, 3, renormalize=True, scale=2.0)     # the tie of experts 0 and 3 goes to 0
    assert ids.tolist() == [[1, 2, 0]] and np.allclose(w, 2 * np.array([[4, 2, 1]]) / 7, rtol=1e-15)


def test_route_bias_moves_the_choice_and_not_the_weight():
    x = np.array([[0.0, 0.0, 2.0]])
    ids, w = moe.route(x, 1, score="sigmoid", bias=np.array([0.0, 1.0, 0.0]), renormalize=False)
    assert ids.tolist() == [[1]] and w[0, 0] == 0.5


def test_route_groups():
    x = np.array([[3.0, 0.0, 2.0, 2.5]])                      # best expert in group 0, best pair in group 1
    assert moe.route(x, 1, n_groups=2, group_score="max", renormalize=False)[0].tolist() == [[0]]
    assert moe.route(x, 1, score="sigmoid", n_groups=2, group_score="top2", renormalize=False)[0].tolist() == [[3]]


def test_route_missing_and_broken_rows():
    inf = np.inf
    x = np.array([[-inf, 1.0, -inf], [-inf, -inf, -inf], [0.0, np.nan, 0.0], [0.0, inf, 0.0]])
    ids, w = moe.route(x, 2)
    assert ids.tolist() == [[1, -1], [-1, -1], [-1, -1], [-1, -1]]
    assert w[0].tolist() == [1.0, 0.0] and w[1].tolist() == [0.0, 0.0] and np.isnan(w[2:]).all()


def test_plan_by_hand():
    offsets, order, slots = moe.plan([[2, 0], [0, -1], [2, 9]], 3)
    assert offsets.tolist() == [0, 2, 2, 4]
    assert order.tolist() == [1, 2, 0, 4, -1, -1]
    assert slots.tolist() == [2, 0, 1, -1, 3, -1]


@pytest.mark.parametrize("E,k,T", [(1, 1, 5), (7, 3, 40), (64, 8, 100)])
def test_plan_is_a_grouping(E, k, T):
    rng = np.random.default_rng(E)
    ids = rng.integers(-1, E + 1, (T, k))
    offsets, order, slots = moe.plan(ids, E)
    held = (ids.reshape(-1) >= 0) & (ids.reshape(-1) < E)
    assert offsets[0] == 0 and offsets[-1] == held.sum() and (order[offsets[-1]:] == -1).all()
    for e in range(E):
        mine = order[offsets[e]: offsets[e + 1]]
        assert (ids.reshape(-1)[mine] == e).all() and (np.diff(mine) > 0).all()
        assert (slots[mine] == np.arange(offsets[e], offsets[e + 1])).all()
    assert (slots[~held] == -1).all()


def test_swiglu_and_combine_by_hand():
    x = np.array([[0.0, 1.0, -200.0, 5.0, 2.0, 3.0]])
    assert np.allclose(moe.swiglu(x), [[0.0, 2.0 / (1.0 + np.exp(-1.0)), 0.0]], rtol=1e-15, atol=1e-80)
    y = np.array([[1.0, 2.0], [10.0, 20.0]])
    out, mag = moe.combine(y, [[1, -1], [0, 1]], [[0.5, 9.0], [1.0, -1.0]], add=np.ones((2, 2)))
    assert out.tolist() == [[6.0, 11.0], [-8.0, -17.0]] and mag.tolist() == [[6.0, 11.0], [12.0, 23.0]]
    assert np.isnan(moe.combine(y, [[-1]], [[np.nan]])[0]).all()


def test_gemm_takes_each_experts_rows_and_scales():
    from gemm_check import exact_operand

    import oracle
    E, N, K, k, T = 3, 128, 256, 2, 5
    ids = np.array([[0, 2], [2, 0], [2, -1], [0, 2], [2, 2]])
    offsets, order, slots = moe.plan(ids, E)
    for scheme in ("fp8_row", "fp8_block128"):
        a = exact_operand(scheme, "activation", T, K, 1)
        w = exact_operand(scheme, "weight", E * N, K, 2)
        A, W = oracle.dequant_exact(a), oracle.dequant_exact(w).reshape(E, N, K)
        C, mag = moe.gemm(a, w, offsets, order, k, True)
        for t in range(T):
            for j in range(k):
                p = slots[t * k + j]
                if p >= 0:
                    assert np.array_equal(C[p], W[ids[t, j]] @ A[t])
                    assert np.array_equal(mag[p], np.abs(W[ids[t, j]]) @ np.abs(A[t]))
