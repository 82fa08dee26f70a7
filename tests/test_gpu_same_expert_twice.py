"""The layer's backward on a finished choice that names an expert twice for a token: the
logit's gradient is the sum over its slots, as in moe_unpermute_backward."""
import numpy as np
import pytest
import torch

from block_cases import BF, assert_within, gen, n64, randn
from mixture_experts_layer_dispatch_amd import binding as B
from oracle.ffn import d_logits_dense

HALF = 2.0 ** -24


def test_the_oracle_adds_up():
    idx = np.array([[2, 0, 2], [1, 1, 1]])
    got = d_logits_dense(idx, np.array([[1.0, 2.0, 4.0], [1.0, 2.0, 4.0]]), 4)
    np.testing.assert_array_equal(got, [[2, 0, 5, 0], [0, 7, 0, 0]])


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(7, 3, 3), (40, 70, 8), (20, 5, 2)])
def test_the_logit_gradient_of_an_expert_named_twice(T, E, k):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    H = I = 128
    cfg = B.Config(T=T, H=H, I=I, E=E, k=k)
    g = gen(T)
    x, dy = randn(g, (T, H), BF), randn(g, (T, H), BF)
    weights = {"w_gate": randn(g, (E, I, H), BF, H ** -0.5), "w_up": randn(g, (E, I, H), BF, H ** -0.5),
               "w_down": randn(g, (E, H, I), BF, I ** -0.5)}
    ws, sched, saved = B.alloc_workspace(cfg), B.alloc_schedule(cfg), B.alloc_saved(cfg)
    sched["topk_idx"].copy_(torch.randint(0, E, (T, k), generator=g, device="cuda"))
    sched["topk_idx"][0] = E - 1
    sched["topk_w"].copy_(torch.rand(T, k, generator=g, device="cuda").softmax(1))
    B.moe_schedule_from_topk(cfg, sched, ws)
    y, dx, grads = torch.empty_like(x), torch.empty_like(x), B.alloc_grads(cfg)
    dw, dl = torch.empty(T, k, device="cuda"), torch.full((T, E), float("nan"), device="cuda")
    B.moe_forward(cfg, sched, x, weights, y, saved, ws)
    B.moe_backward(cfg, sched, saved, x, weights, dy, dx, grads, dw, dl, ws)
    assert B.moe_check_device_error(ws) == 0
    w, d, idx = n64(sched["topk_w"]), n64(dw), sched["topk_idx"].cpu().numpy()
    sel = w * (d - (w * d).sum(1, keepdims=True))
    mag = w * (np.abs(d) + (w * np.abs(d)).sum(1, keepdims=True))
    # k products and sums, a difference and a product, and the sum over the slots
    tol = (2 * k + 4) * HALF * d_logits_dense(idx, mag, E)
    assert_within("d_logits", dl, d_logits_dense(idx, sel, E), tol)
