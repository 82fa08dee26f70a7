"""Pins of the reference of routing with scores, norm and 4-bit linear: hand-worked
cases, brute force and central differences in 64 bits."""
import itertools

import numpy as np
import pytest

from oracle import around, routing


def test_route_by_hand():
    # sigmoid(0) = 1/2; the bias decides the choice but not the weights
    l = np.array([[0.0, 0.0, np.log(3.0), -np.log(3.0)]])                 # scores 1/2, 1/2, 3/4, 1/4
    idx, w, s = around.route(l, 2, "sigmoid")
    np.testing.assert_array_equal(idx, [[2, 0]])                         # the tie goes to expert 0
    np.testing.assert_allclose(w, [[0.6, 0.4]])
    np.testing.assert_allclose(s, [[0.5, 0.5, 0.75, 0.25]])
    idx, w, _ = around.route(l, 2, "sigmoid", bias=[0, 0.01, -0.5, 0.6], renorm=False, scale=2.0)
    np.testing.assert_array_equal(idx, [[3, 1]])
    np.testing.assert_allclose(w, [[0.5, 1.0]])
    # groups of two: {1/2, 1/2} sums to 1 as {3/4, 1/4} does; the tie goes to the lower group
    idx, _, _ = around.route(l, 2, "sigmoid", n_group=2, topk_group=1, group_top=2)
    np.testing.assert_array_equal(idx, [[0, 1]])
    idx, _, _ = around.route(l, 2, "sigmoid", n_group=2, topk_group=1, group_top=1)
    np.testing.assert_array_equal(idx, [[2, 3]])
    # what leaves nothing: lowest experts, weights 0; infinite ones share
    idx, w, s = around.route(np.full((1, 4), -np.inf), 2)
    np.testing.assert_array_equal(idx, [[0, 1]])
    assert not w.any() and not s.any()
    idx, w, s = around.route([[0.0, np.inf, 1.0, np.inf]], 3, renorm=False)
    np.testing.assert_array_equal(idx, [[1, 3, 2]])
    np.testing.assert_allclose(w, [[0.5, 0.5, 0.0]])


def test_route_without_extras_is_the_layers_routing():
    l = np.random.default_rng(3).standard_normal((20, 12)).astype(np.float32)
    idx, w, s = around.route(l, 4)
    ref_idx, ref_w = routing.route(l, 4)
    np.testing.assert_array_equal(idx, ref_idx)
    np.testing.assert_allclose(w, ref_w, rtol=1e-6)
    np.testing.assert_allclose(s.sum(1), 1)
    np.testing.assert_allclose(around.route(l, 12, renorm=False, scale=2.5)[1].sum(1), 2.5)


def test_route_groups_against_all_subsets():
    rng = np.random.default_rng(5)
    l, b = rng.standard_normal((15, 12)), rng.standard_normal(12) * 0.1
    idx, _, s = around.route(l, 3, "sigmoid", b, n_group=4, topk_group=2, group_top=2)
    c = s + b
    for t in range(15):
        g = [sum(sorted(c[t, 3 * i:3 * i + 3])[1:]) for i in range(4)]
        best = max(itertools.combinations(range(4), 2), key=lambda p: g[p[0]] + g[p[1]])
        members = [3 * i + j for i in best for j in range(3)]
        top = max(itertools.permutations(members, 3), key=lambda p: (c[t, p[0]], c[t, p[1]], c[t, p[2]]))
        np.testing.assert_array_equal(idx[t], top)


def _diff(f, x, eps=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + eps
        hi = f()
        x[i] = old - eps
        g[i] = (hi - f()) / (2 * eps)
        x[i] = old
    return g


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dense", [True, False])
def test_route_backward_by_differences(score, renorm, dense):
    rng = np.random.default_rng(7)
    l, dw, ds = rng.standard_normal((4, 6)), rng.standard_normal((4, 3)), rng.standard_normal((4, 6))
    idx = around.route(l, 3, score)[0]

    def loss():
        s = around.scores(l, score)
        w = np.take_along_axis(s, idx, 1)
        w = 1.7 * (w / w.sum(1, keepdims=True) if renorm else w)
        return (w * dw).sum() + ((s * ds).sum() if dense else 0)

    got = around.route_backward(l, idx, dw, score, renorm, 1.7, ds if dense else None)
    np.testing.assert_allclose(got, _diff(loss, l), atol=1e-8)


def test_route_backward_of_tables_and_of_nothing():
    l, dw = np.random.default_rng(8).standard_normal((2, 5)), np.ones((2, 3)) * [[1.0], [2.0]]
    one = around.route_backward(l, np.array([[1, 3, 3]] * 2), dw, "sigmoid", False)
    two = around.route_backward(l, np.array([[1, 3, 9]] * 2), dw, "sigmoid", False)
    np.testing.assert_allclose(one[:, 3], 2 * two[:, 3])
    assert not around.route_backward(np.full((1, 4), -np.inf), np.array([[0, 1]]), np.ones((1, 2))).any()


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_by_differences(kind):
    rng = np.random.default_rng(9)
    h, gamma, beta, dy, dt = (rng.standard_normal(s) for s in ((3, 5), 5, 5, (3, 5), (3, 5)))
    if kind == "rms":
        beta = None
    y, mean, rstd = around.norm(h, gamma, beta, kind)
    if kind == "layer":
        np.testing.assert_allclose(((y - beta) / gamma).mean(1), 0, atol=1e-12)
    np.testing.assert_allclose((((y - (0 if beta is None else beta)) / gamma) ** 2).mean(1), 1, atol=1e-4)

    def loss():
        return (around.norm(h, gamma, beta, kind)[0] * dy).sum() + (h * dt).sum()

    dx, dgamma, dbeta = around.norm_backward(h, gamma, mean, rstd, dy, kind, dt)
    np.testing.assert_allclose(dx, _diff(loss, h), atol=1e-8)
    np.testing.assert_allclose(dgamma, _diff(loss, gamma), atol=1e-8)
    if beta is not None:
        np.testing.assert_allclose(dbeta, _diff(loss, beta), atol=1e-8)


def test_w4_by_hand():
    codes = np.array([[0x80, 0x9F], [0x07, 0xF1]], np.uint8)              # [N, K / 2]
    np.testing.assert_array_equal(around.w4_codes(codes), [[0, 8, 15, 9], [7, 0, 1, 15]])
    scales = np.array([[0.5, 2.0], [1.0, 0.25]])                         # [K / 2, N]
    np.testing.assert_allclose(around.w4_weights(codes, scales), [[-4, 0, 7, 1], [-2, -16, -1.75, 1.75]])
    zeros = np.array([[0, 7], [15, 1]])
    w = around.w4_weights(codes, scales, zeros)
    np.testing.assert_allclose(w, [[0, 4, 0, -6], [0, -14, 0, 3.5]])
    x = np.array([[1.0, 2, 3, 4], [0, -1, 0, 1]])
    y, _, mag = around.linear_w4(x, codes, scales, zeros, bias=[1.0, -100], activation="relu", residual=np.ones((2, 2)))
    np.testing.assert_allclose(y, [[1, 1], [1, 1]])                      # 8 - 24 + 1, -28 + 14 - 100, -4 - 6 + 1, ...
    np.testing.assert_allclose(mag, [[33, 142], [11, 117.5]])
    y, _, _ = around.linear_w4(x, np.stack([codes] * 2), np.stack([scales] * 2), offsets=[0, 1, 2])
    np.testing.assert_allclose(y, x @ around.w4_weights(codes, scales).T)


@pytest.mark.parametrize("zeros", [False, True])
def test_w4_quantize(zeros):
    rng = np.random.default_rng(11)
    exact = lambda a: a.astype(np.float64)                               # noqa: E731
    w = rng.standard_normal((3, 64))
    w[1, :32] = 0
    w[2, 32:] = np.abs(w[2, 32:])
    q, s, z = around.w4_quantize(w, 32, exact, zeros)
    packed = (q[..., 0::2] | q[..., 1::2] << 4).astype(np.uint8)
    back = around.w4_weights(packed, s, z)
    step = np.repeat(s.T, 32, 1)
    # within half a step (and, with a rounded zero point, half a step more at the ends)
    assert np.all(np.abs(back - w) <= step * (1.0 if zeros else 0.5) + 1e-6)
    assert not back[1, :32].any()
    # weights that codes stand for come back
    codes = rng.integers(1, 16, (3, 64))
    codes[:, ::32], codes[:, 1::32] = 15, (0 if zeros else 1)
    q2, s2, z2 = around.w4_quantize((codes - 8) * 0.25, 32, exact, zeros)
    np.testing.assert_array_equal(q2, codes)
    assert np.all(s2 == 0.25) and (z2 is None or np.all(z2 == 8))
