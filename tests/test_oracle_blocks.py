"""The 64-bit reference of the building blocks (oracle.blocks): its gradients
against central differences of its forward."""
import numpy as np
import pytest

from oracle import blocks


def _diff(f, a, h=1e-5):
    """Central differences of the scalar f() in every element of a (changed in place)."""
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        old = a[i]
        a[i] = old + h
        up = f()
        a[i] = old - h
        down = f()
        a[i] = old
        g[i] = (up - down) / (2 * h)
    return g


@pytest.mark.parametrize("name", blocks.ACTS)
@pytest.mark.parametrize("offsets", [None, [0, 3, 3, 5]])
def test_linear_gradients_are_those_of_the_forward(name, offsets):
    rng = np.random.default_rng(7)
    M, N, K, E = 6, 4, 5, 3
    lead = () if offsets is None else (E,)
    x, w = rng.standard_normal((M, K)), rng.standard_normal((*lead, N, K))
    b, dy = rng.standard_normal((*lead, N)), rng.standard_normal((M, N))
    live = slice(0, M if offsets is None else offsets[-1])

    def loss():
        return float((blocks.linear(x, w, b, None, name, offsets)[0] * dy)[live].sum())

    z = blocks.linear(x, w, b, None, name, offsets)[1]
    g = blocks.linear_backward(x, w, np.nan_to_num(z), dy, name, offsets)
    np.testing.assert_allclose(np.nan_to_num(g["dx"]), _diff(loss, x), rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(g["dw"], _diff(loss, w), rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(g["db"], _diff(loss, b), rtol=1e-6, atol=1e-7)


def test_unpermute_gradients_are_those_of_the_forward():
    rng = np.random.default_rng(8)
    T, k, H, E = 5, 2, 3, 4
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    logits = rng.standard_normal((T, E))
    row = rng.permutation(T * k)
    o, dy, res = rng.standard_normal((T * k, H)), rng.standard_normal((T, H)), rng.standard_normal((T, H))

    def weights():
        v = np.exp(np.take_along_axis(logits, idx, 1))
        return v / v.sum(1, keepdims=True)

    def loss():
        return float((blocks.unpermute(o, row, weights(), res) * dy).sum())

    do, dw, dl = blocks.unpermute_backward(o, dy, row, weights(), idx, E)
    np.testing.assert_allclose(do, _diff(loss, o), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(dl, _diff(loss, logits), rtol=1e-6, atol=1e-8)
    w = weights()
    np.testing.assert_allclose(dw, _diff(lambda: float((blocks.unpermute(o, row, w) * dy).sum()), w), rtol=1e-6,
                               atol=1e-8)


def test_permute_backward_is_the_transpose():
    rng = np.random.default_rng(9)
    T, k, H = 4, 3, 2
    row = rng.permutation(T * k)
    x, d = rng.standard_normal((T, H)), rng.standard_normal((T * k, H))
    assert np.isclose((blocks.permute(x, row, k) * d).sum(), (x * blocks.permute_backward(d, row, k)).sum())
