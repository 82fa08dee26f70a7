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



# one wrong argument each: a missing or misaligned buffer
REQUIRED = [(c, n) for c, (bufs, reads) in CALLS.items() for n in bufs + reads if n not in ("residual", "d_logits")]


@pytest.mark.parametrize("name,arg", REQUIRED)
def test_a_buffer_that_is_missing(name, arg):
    assert _call(name, **{arg: None}) == B.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("name,arg", [(c, n) for c, (bufs, reads) in CALLS.items() for n in bufs + reads])
def test_a_buffer_that_is_not_aligned(name, arg):
    by = 2 if arg in (*SCHED, "dw", "d_logits") else 8     # 4 bytes of indices and fp32 values, 16 of rows
    assert _call(name, **{arg: ADDR[arg] + by}) == B.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("name", list(CALLS))
def test_types_configs_schedules_workspaces(name):
    for dtype in (-1, 3):
        assert _call(name, dtype=dtype) == B.MOE_ERR_INVALID_ARG
    assert _call(name, sched=False) == B.MOE_ERR_INVALID_ARG
    assert _call(name, with_cfg=False) == B.MOE_ERR_INVALID_ARG
    for change in (dict(H=100), dict(H=0), dict(T=0), dict(k=0), dict(k=5), dict(E=0), dict(E=1025), dict(I=0)):
        cfg = B.Config(**{**dict(T=8, H=128, I=128, E=4, k=2), **change})
        assert _call(name, cfg=cfg) == B.MOE_ERR_INVALID_ARG
    assert _call(name, ws=None) == B.MOE_ERR_WORKSPACE
    assert _call(name, ws=ADDR["ws"] + 128) == B.MOE_ERR_WORKSPACE
    assert _call(name, ws_bytes=255) == B.MOE_ERR_WORKSPACE


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


@pytest.mark.parametrize("name,arg", [(c, n) for c, args in LIN_CALLS.items() for n in args
                                      if n not in ("bias", "residual") and (c, n) != ("moe_linear_forward", "z")
                                      and n not in ("dx", "dw", "db")])
def test_a_buffer_of_linear_that_is_missing(name, arg):
    assert _linear(name, **{arg: None}) == B.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("name,arg", [(c, n) for c, args in LIN_CALLS.items() for n in args])
def test_a_buffer_of_linear_that_is_not_aligned(name, arg):
    assert _linear(name, **{arg: LIN[arg] + (2 if arg == "offsets" else 8)}) == B.MOE_ERR_INVALID_ARG


def test_what_linear_may_be_given_without():
    assert _linear("moe_linear_forward", bias=None, residual=None, z=None) == PASSES
    for gone in (("dx", "w"), ("dw", "x"), ("db",), ("dx", "dw", "w", "x")):
        assert _linear("moe_linear_backward", **{n: None for n in gone}) == PASSES
    assert _linear("moe_linear_backward", dx=None, dw=None, db=None) == B.MOE_ERR_INVALID_ARG
    for name in LIN_CALLS:
        assert _linear(name, E=0, offsets=None) == PASSES
        assert _linear(name, E=0) == B.MOE_ERR_INVALID_ARG
