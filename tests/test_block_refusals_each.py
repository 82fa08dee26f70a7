"""Refusals of permute and unpermute at the C entry points, one wrong argument
at a time: every other buffer has an address of its own, so that no other check
can refuse the call.  Without a GPU a call that passes its checks ends with
MOE_ERR_UNSUPPORTED_DEVICE; with one these calls are not made, since only the
refused ones would be safe."""
import pytest
import torch

from mixture_experts_layer_dispatch_amd import binding as B

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="calls that pass the checks would run")

NAMES = ["topk_idx", "topk_w", "row_of_slot", "x", "xs", "dxs", "dx", "o", "residual", "y", "dy", "do", "dw",
         "d_logits", "ws"]
ADDR = {n: (i + 1) << 20 for i, n in enumerate(NAMES)}                 # never dereferenced
SCHED = ("topk_idx", "topk_w", "row_of_slot")
# the buffers of each call in the order of its arguments, and the schedule's arrays it reads
CALLS = {"moe_permute_forward": (["x", "xs"], ["row_of_slot"]),
         "moe_permute_backward": (["dxs", "dx"], ["row_of_slot"]),
         "moe_unpermute_forward": (["o", "residual", "y"], ["row_of_slot", "topk_w"]),
         "moe_unpermute_backward": (["o", "dy", "do", "dw", "d_logits"], ["row_of_slot", "topk_w", "topk_idx"])}
PASSES = B.MOE_ERR_UNSUPPORTED_DEVICE


def _call(name, cfg=None, dtype=0, sched=True, ws_bytes=256, with_cfg=True, **addr):
    """Status of the call with the named addresses changed (None: a null pointer)."""
    a = {**ADDR, **addr}
    cfg = (cfg or B.Config(T=8, H=128, I=128, E=4, k=2)).c() if with_cfg else None
    reads = CALLS[name][1]
    s = B.moe_sched(**{n: a[n] for n in reads}) if sched else None
    return getattr(B.lib(), name)(cfg, s, dtype, *[a[n] for n in CALLS[name][0]], a["ws"], ws_bytes, None)


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_the_calls_pass_as_they_are(name, dtype):
    assert _call(name, dtype=dtype) == PASSES
    optional = {"moe_unpermute_forward": "residual", "moe_unpermute_backward": "d_logits"}.get(name)
    if optional:
        assert _call(name, dtype=dtype, **{optional: None}) == PASSES
    if name == "moe_unpermute_backward":                  # topk_idx is read for d_logits only
        assert _call(name, dtype=dtype, d_logits=None, topk_idx=None) == PASSES
    if name == "moe_unpermute_forward":                   # the one pair that may be the same
        assert _call(name, dtype=dtype, residual=ADDR["y"]) == PASSES


# an output that is another buffer of the call
TWICE = [(c, out, other) for c, outs in (("moe_permute_forward", ["xs"]), ("moe_permute_backward", ["dx"]),
                                         ("moe_unpermute_forward", ["y"]),
                                         ("moe_unpermute_backward", ["do", "dw", "d_logits"]))
         for out in outs for other in CALLS[c][0] + CALLS[c][1] if out != other and (out, other) != ("y", "residual")]


@pytest.mark.parametrize("name,out,other", TWICE)
def test_an_output_is_no_other_buffer(name, out, other):
    assert _call(name, **{out: ADDR[other]}) == B.MOE_ERR_INVALID_ARG


# ------------------------------------------------------------------ linear
LIN = {n: (i + 32) << 20 for i, n in enumerate(["offsets", "x", "w", "bias", "residual", "y", "z", "dy", "dx", "dw",
                                                "db", "ws"])}
LIN_CALLS = {"moe_linear_forward": ["offsets", "x", "w", "bias", "residual", "y", "z"],
             "moe_linear_backward": ["offsets", "x", "w", "z", "dy", "dx", "dw", "db"]}


def _linear(name, E=4, **addr):
    a = {**LIN, **addr}
    c = B.moe_linear_config(64, 128, 256, E, 0, B.ACTS["silu"], 0)
    return getattr(B.lib(), name)(c, *[a[n] for n in LIN_CALLS[name]], a["ws"], 1 << 40, None)


LIN_TWICE = [(c, out, other) for c, outs in (("moe_linear_forward", ["y", "z"]),
                                             ("moe_linear_backward", ["dx", "dw", "db"]))
             for out in outs for other in LIN_CALLS[c] if out != other and (out, other) != ("y", "residual")]


@pytest.mark.parametrize("name,out,other", LIN_TWICE)
def test_an_output_of_linear_is_no_other_buffer(name, out, other):
    assert _linear(name) == PASSES
    assert _linear(name, **{out: LIN[other]}) == B.MOE_ERR_INVALID_ARG
    assert _linear("moe_linear_forward", residual=LIN["y"]) == PASSES
