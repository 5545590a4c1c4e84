"""The plain top-k routing of the tests against facts that do not come from it."""
import numpy as np
import pytest

import topk_reference as ref


def test_softmax_and_sigmoid_scores():
    z = np.array([0.0, np.log(3.0), -np.inf])
    assert np.allclose(ref.scores64(z, "softmax"), [0.25, 0.75, 0])
    assert np.allclose(ref.scores64(z, "sigmoid"), [0.5, 0.75, 0])


def test_hand_example():
    """Eight experts in four groups; the bias moves the choice but not the weights."""
    z = np.log(np.array([[0.5, 0.1, 0.4, 0.4, 0.05, 0.05, 0.9, 0.01]]) / (1 - np.array(
        [[0.5, 0.1, 0.4, 0.4, 0.05, 0.05, 0.9, 0.01]])))
    # group values 0.6, 0.8, 0.1, 0.91: groups 1 and 3 take part; 2 and 3 tie
    _, ids, w = ref.route(z, 2, "sigmoid", None, 4, 2, renorm=False)
    assert ids.tolist() == [[6, 2]] and np.allclose(w, [[0.9, 0.4]])
    bias = np.array([1.0, 0, 0, 0, 0, 0, 0, 0])
    _, ids, w = ref.route(z, 2, "sigmoid", bias, 4, 2, renorm=True)   # groups 0 (1.6) and 3
    assert ids.tolist() == [[0, 6]] and np.allclose(w, [[0.5 / 1.4, 0.9 / 1.4]])


def test_masked_rows_and_ties():
    z = np.array([[-np.inf] * 4, [1.0, -np.inf, 1.0, np.nan]])
    gates, ids, w = ref.route(z, 3)
    assert ids.tolist() == [[-1, -1, -1], [0, 2, -1]]
    assert np.allclose(w, [[0, 0, 0], [0.5, 0.5, 0]]) and np.allclose(gates[1], [0.5, 0, 0.5, 0])


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(kind, renorm):
    rng = np.random.default_rng(5)
    T, E, k, h = 3, 11, 4, 1e-5
    z = rng.standard_normal((T, E))
    _, ids, _ = ref.route(z, k, kind)
    ids[2, 3] = -1
    dw = rng.standard_normal((T, k))
    got, _ = ref.backward(z, ids, dw, kind, renorm, 1.7)

    def loss(zz):
        s = 0.0
        for t in range(T):
            live = [i for i in range(k) if ids[t, i] >= 0]
            s += (ref.weights64(zz[t], ids[t, live], kind, renorm, 1.7) * dw[t, live]).sum()
        return s

    for t in range(T):
        for e in range(E):
            d = np.zeros_like(z)
            d[t, e] = h
            # central differences: error of order h^2 and 2^-52 / h
            assert abs((loss(z + d) - loss(z - d)) / (2 * h) - got[t, e]) < 1e-8
