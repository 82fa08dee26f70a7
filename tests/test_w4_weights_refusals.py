"""Buffers of 4-bit weights are made only for a config that the product takes."""
import pytest

from mixture_experts_layer_dispatch_amd import binding as B


@pytest.mark.parametrize("change", [dict(group=0), dict(group=48), dict(group=256), dict(K=100), dict(K=0), dict(N=12),
                                    dict(N=0), dict(E=-1), dict(E=1025), dict(K=1 << 17), dict(N=1 << 17), dict(act="tanh"),
                                    dict(K=(1 << 32) + 128)])
@pytest.mark.parametrize("zeros", [False, True])
def test_refused(change, zeros):
    wc = B.LinearW4Config(**{**dict(M=1, N=16, K=256, group=128), **change})
    with pytest.raises((B.MoEError, ValueError)):
        B.alloc_linear_w4_weights(wc, zeros, device="cpu")


def test_shapes():
    q = B.alloc_linear_w4_weights(B.LinearW4Config(M=1, N=16, K=256, E=3, group=64), True, device="cpu")
    assert {n: tuple(t.shape) for n, t in q.items()} == {"codes": (3, 16, 128), "scales": (3, 4, 16), "zeros": (3, 4, 16)}
