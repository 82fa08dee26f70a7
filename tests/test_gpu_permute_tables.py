"""Schedule tables built by the caller: an expert chosen twice by a token, and
experts outside the layer's."""
import numpy as np
import pytest
import torch

from block_cases import BF, F32, FP, assert_within, gen, n64, randn, schedule, sum_err
from mixture_experts_layer_dispatch_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _backward(cfg, sched, ws, o, dy):
    do, dw = torch.full_like(o, -77.0), torch.full((cfg.T, cfg.k), -77.0, device="cuda")
    dl = torch.full((cfg.T, cfg.E), -77.0, device="cuda")
    B.moe_unpermute_backward(cfg, sched, o, dy, do, dw, ws, d_logits=dl)
    return do, dw, dl


# one wave a token, then several; one batch of slots, then several
SHAPES = [(20, 9, 4, 128), (20, 9, 4, 1152), (11, 40, 17, 256), (7, 200, 12, 2048)]


@pytest.mark.parametrize("dtype", [BF, FP, F32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,E,k,H", SHAPES)
def test_an_expert_chosen_twice_gets_both_gradients(T, E, k, H, dtype):
    """Its logit stands in the softmax twice: d_logit is the sum over its slots."""
    cfg, sched, ws = schedule(51, T, E, k, H)
    g = gen(52)
    o, dy = randn(g, (T * k, H), dtype), randn(g, (T, H), dtype)
    plain = _backward(cfg, sched, ws, o, dy)
    idx = sched["topk_idx"].clone()
    idx[::2, 1] = idx[::2, 0]                               # every other token: slots 0 and 1 (and the last)
    idx[::4, -1] = idx[::4, 0]
    sched["topk_idx"] = idx
    do, dw, dl = _backward(cfg, sched, ws, o, dy)
    assert torch.equal(do, plain[0]) and torch.equal(dw, plain[1])
    assert torch.equal(dl[1::2], plain[2][1::2])
    w, w64 = sched["topk_w"], n64(sched["topk_w"])
    # from the dw that was written: w (dw - sum w dw), k + 4 roundings of those terms, added over the slots
    d = n64(dw)
    share = w64 * (d - (w64 * d).sum(1, keepdims=True))
    serr = sum_err(k + 4, w64 * (np.abs(d) + (w64 * np.abs(d)).sum(1, keepdims=True)))
    ref, tol = np.zeros((T, E)), np.full((T, E), 1e-37)
    t = np.arange(T)[:, None]
    np.add.at(ref, (t, idx.cpu().numpy()), share)
    np.add.at(tol, (t, idx.cpu().numpy()), serr + 2.0 ** -22 * np.abs(share))
    assert_within("dl", dl, ref, tol)
    assert w.shape == (T, k) and B.moe_check_device_error(ws) == 0


@pytest.mark.parametrize("T,E,k,H", SHAPES)
def test_experts_outside_the_layer_are_skipped_and_reported(T, E, k, H):
    cfg, sched, ws = schedule(53, T, E, k, H)
    g = gen(54)
    o, dy = randn(g, (T * k, H), BF), randn(g, (T, H), BF)
    plain = _backward(cfg, sched, ws, o, dy)
    assert B.moe_check_device_error(ws) == 0
    good = sched["topk_idx"]
    for bad in (E, -1, 1 << 30):
        idx = good.clone()
        idx[3, 2] = bad
        do, dw, dl = _backward(cfg, {**sched, "topk_idx": idx}, ws, o, dy)
        assert B.moe_check_device_error(ws) == B.DEVERR_BAD_EXPERT
        assert B.moe_check_device_error(ws) == 0            # read and cleared
        want = plain[2].clone()
        want[3, good[3, 2].long()] = 0
        assert torch.equal(dl, want) and torch.equal(do, plain[0]) and torch.equal(dw, plain[1])
        B.moe_unpermute_backward(cfg, {**sched, "topk_idx": idx}, o, dy, do, dw, ws)      # not read
        assert B.moe_check_device_error(ws) == 0
