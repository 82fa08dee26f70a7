"""A table whose choice names experts outside the layer, through the layer itself.  A slot
without a row adds nothing: y, dx and the weights' gradients are those of the same table with
a weight of zero in that slot, for one expert a token (whose outputs the products write
themselves) as for several."""
import pytest
import torch

from block_cases import BF, F32, gen, randn
from mixture_experts_layer_dispatch_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def run(cfg, weights, idx, w, x, dy):
    ws, sched, saved = B.alloc_workspace(cfg), B.alloc_schedule(cfg), B.alloc_saved(cfg)
    sched["topk_idx"].copy_(idx)
    sched["topk_w"].copy_(w)
    B.moe_schedule_from_topk(cfg, sched, ws)
    flags = [B.moe_check_device_error(ws)]
    y = torch.full_like(x, float("nan"))
    B.moe_forward(cfg, sched, x, weights, y, saved, ws)
    flags.append(B.moe_check_device_error(ws))
    if cfg.precision == B.PREC_MXFP4:
        return flags, {"y": y}
    dx, grads = torch.full_like(x, float("nan")), B.alloc_grads(cfg)
    dw = torch.full((cfg.T, cfg.k), float("nan"), device="cuda")
    dl = torch.full((cfg.T, cfg.E), float("nan"), device="cuda")
    B.moe_backward(cfg, sched, saved, x, weights, dy, dx, grads, dw, dl, ws)
    flags.append(B.moe_check_device_error(ws))
    return flags, {"y": y, "dx": dx, "dw": dw, "d_logits": dl, **grads}


@pytest.mark.parametrize("k", [1, 2])
@pytest.mark.parametrize("T,macrobatch,E,H,I", [(48, 0, 9, 128, 128), (48, 16, 9, 384, 128), (600, 0, 3, 256, 256),
                                                (5, 0, 4, 128, 256)])
@pytest.mark.parametrize("precision", [B.PREC_BF16, B.PREC_MXFP8, B.PREC_MXFP4])
@pytest.mark.parametrize("n_shared", [0, 1])
def test_a_slot_without_a_row_is_a_slot_of_weight_zero(T, macrobatch, E, H, I, k, precision, n_shared):
    cfg = B.Config(T=T, H=H, I=I, E=E, k=k, macrobatch=macrobatch, precision=precision, n_shared=n_shared)
    g = gen(T + E)
    x, dy = randn(g, (T, H), BF), randn(g, (T, H), BF)
    weights = {"w_gate": randn(g, (E, I, H), BF, H ** -0.5), "w_up": randn(g, (E, I, H), BF, H ** -0.5),
               "w_down": randn(g, (E, H, I), BF, I ** -0.5)}
    if n_shared:
        weights.update(s_gate=randn(g, (I, H), BF, H ** -0.5), s_up=randn(g, (I, H), BF, H ** -0.5),
                       s_down=randn(g, (H, I), BF, I ** -0.5))
    if precision == B.PREC_MXFP8:
        mx = B.alloc_weights_mx(cfg)
        B.moe_quantize_weights_mxfp8(cfg, weights, mx)
        weights["mx"] = mx
    if precision == B.PREC_MXFP4:
        mx = B.alloc_weights_mx4(cfg)
        B.moe_quantize_weights_mxfp4(cfg, weights, mx)
        weights["mx4"] = mx
    idx = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.int()
    w = torch.rand(T, k, generator=g, device="cuda") + 0.5
    missing = torch.rand(T, k, generator=g, device="cuda") < 0.2
    missing[0, 0] = missing[T - 1, k - 1] = missing[T // 2, 0] = True
    odd = torch.tensor([-1, E, 1 << 30, -(1 << 31)], dtype=torch.int32, device="cuda")
    bad = torch.where(missing, odd[torch.arange(T, device="cuda") % 4].unsqueeze(1), idx)
    zeroed = torch.where(missing, 0.0, w)
    flags, got = run(cfg, weights, bad, w, x, dy)
    assert flags == [B.DEVERR_BAD_EXPERT, *[B.DEVERR_BAD_ROW] * (len(flags) - 1)]
    clean, ref = run(cfg, weights, idx, zeroed, x, dy)
    assert clean == [0] * len(clean)
    # (a row's sums over H and I do not depend on its place in a tile)
    assert torch.equal(got["y"], ref["y"])
    if k == 1 and not n_shared:
        assert (got["y"][missing[:, 0]] == 0).all()
    if precision == B.PREC_MXFP4:
        return
    assert torch.equal(got["dx"], ref["dx"])
    assert (got["dw"][missing] == 0).all() and torch.equal(got["dw"][~missing], ref["dw"][~missing])
    assert got["d_logits"].isfinite().all()
    for n in ("d_w_gate", "d_w_up", "d_w_down"):
        assert got[n].isfinite().all(), n
        if precision == B.PREC_BF16:
            # the same products in sums of another order: two roundings to bf16 of values that far apart
            a, b = got[n].to(F32), ref[n].to(F32)
            assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-3 * b.abs().amax()).all(), n
