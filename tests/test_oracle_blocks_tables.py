"""The reference's logit gradient for tables that name an expert more than once
a token, against central differences through the softmax over the slots."""
import numpy as np

from oracle import blocks


def test_logit_gradient_of_an_expert_chosen_twice():
    rng = np.random.default_rng(3)
    T, E, k, H = 5, 6, 4, 8
    logits = rng.standard_normal((T, E))
    idx = rng.integers(0, E, (T, k))
    idx[:3, 1] = idx[:3, 0]
    row = rng.permutation(T * k)
    o, dy = rng.standard_normal((T * k, H)), rng.standard_normal((T, H))

    def weights(l):
        v = np.exp(np.take_along_axis(l, idx, 1))
        return v / v.sum(1, keepdims=True)

    dl = blocks.unpermute_backward(o, dy, row, weights(logits), idx, E)[2]
    h = 1e-6
    for t in range(T):
        for e in range(E):
            a, b = logits.copy(), logits.copy()
            a[t, e] += h
            b[t, e] -= h
            f = [(blocks.unpermute(o, row, weights(l)) * dy).sum() for l in (a, b)]
            # h^2 / 6 of a third derivative of order 10, and 2^-52 of a sum of order 100 over 2 h
            assert abs(dl[t, e] - (f[0] - f[1]) / (2 * h)) < 1e-7
