"""The 64-bit forms of the layer operators against worked values and against
differences (no GPU)."""
import numpy as np
import pytest

import layer_reference as ref


def test_unpack_follows_the_word_order():
    # word 0x76543210 little-endian: weight k is nibble k
    w = np.frombuffer(np.array([0x76543210, 0xFEDCBA98], "<u4").tobytes(), np.uint8)
    assert ref.unpack_q4(w, 1, 16).tolist() == [list(range(16))]


def test_linear_worked_value():
    w = np.full((1, 16), 0x98, np.uint8)                       # weights 8, 9, 8, 9, ...
    x = np.ones((1, 32))
    out, _ = ref.linear(w, np.array([[0.5]]), None, 32, x, 1, 32)
    assert out[0, 0] == 0.5 * 16
    out, _ = ref.linear(w, np.array([[0.5]]), np.array([[-1.0]]), 32, x, 1, 32)
    assert out[0, 0] == 0.5 * (8 * 16 + 9 * 16) - 32


def test_route_worked_value():
    l = np.log(np.array([[1.0, 4.0, 2.0, 1.0]]))
    ids, w, counts, loss, grad = ref.route(l, 2, "softmax")
    assert ids.tolist() == [[1, 2]] and np.allclose(w, [[0.5, 0.25]])
    # f = [0, 1/2, 1/2, 0], P = softmax
    assert counts.tolist() == [0, 1, 1, 0] and np.isclose(loss, 4 * (0.5 * 0.5 + 0.5 * 0.25))
    assert np.allclose(grad, [0, 2, 2, 0])
    assert ref.route(l, 3, "softmax")[0].tolist() == [[1, 2, 0]]          # tie: lowest index
    even = ref.route(np.zeros((8, 4)), 4, "softmax")
    assert np.isclose(even[3], 1.0)                                      # perfectly balanced


def test_route_masks_and_limits():
    l = np.array([[0.0, -np.inf, 1.0], [-np.inf] * 3, [np.nan] * 3])
    ids, w, counts, _, _ = ref.route(l, 3, "softmax", mask=np.array([1, 1, 0]))
    assert ids.tolist() == [[2, 0, -1], [-1] * 3, [-1] * 3]
    assert np.all(w[1:] == 0) and counts.tolist() == [1, 0, 1]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_against_differences(score, renormalize):
    rng = np.random.default_rng(5)
    M, E, K = 4, 9, 3
    l = rng.normal(size=(M, E))
    ids, _, _, _, grad = ref.route(l, K, score)
    ids[1] = -1                                                           # an empty token
    dw = rng.normal(size=(M, K))
    args = (ids, score, renormalize, 2.5, dw, 0.7, grad)
    got, _ = ref.route_backward(l, *args)
    h = 1e-6
    for t in range(M):
        for e in range(E):
            up, down = l.copy(), l.copy()
            up[t, e] += h
            down[t, e] -= h
            num = (ref.route_objective(up, *args) - ref.route_objective(down, *args)) / (2 * h)
            assert abs(num - got[t, e]) < 1e-7, (t, e)


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(6)
    M, K, H = 2, 3, 8
    y, w, d = rng.normal(size=(M, K, H)), rng.normal(size=(M, K)), rng.normal(size=(M, H))
    ids = np.array([[0, 1, -1], [5, 2, 0]])
    f = lambda y_, w_: float((ref.combine(y_, w_, ids, 3, None)[0] * d).sum())
    d_y, d_w, _ = ref.combine_backward(d, y, w, ids, 3)
    h = 1e-6
    for at in np.ndindex(M, K):
        up, down = w.copy(), w.copy()
        up[at] += h
        down[at] -= h
        assert abs((f(y, up) - f(y, down)) / (2 * h) - d_w[at]) < 1e-8
    for at in np.ndindex(M, K, H):
        up, down = y.copy(), y.copy()
        up[at] += h
        down[at] -= h
        assert abs((f(up, w) - f(down, w)) / (2 * h) - d_y[at]) < 1e-8
