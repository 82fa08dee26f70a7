"""Sizes that do not fit the C ABI's fields are refused, on the host: cut to
the fields' bits they would be other, valid sizes."""
import pytest
import torch

from mixture_experts_layer_dispatch_amd import binding as B

WRAP = 1 << 32                       # a field's value plus this has the same low 32 bits
SIZES = dict(T=64, H=128, I=128, E=8, k=2, n_shared=1, macrobatch=32, minibatch=16, capacity_rows=128,
             precision=B.PREC_MXFP8, acc_experts=4)


@pytest.mark.parametrize("field", ["M", "N", "K", "E"])
@pytest.mark.parametrize("by", [WRAP, -WRAP, 1 << 31, 1 << 40])
def test_linear_config(field, by):
    sizes = dict(M=64, N=128, K=256, E=4)
    assert B.linear_workspace_size(B.LinearConfig(**sizes)) > 0
    sizes[field] += by
    with pytest.raises(ValueError, match=f"{field}: .* 32 bits"):
        B.linear_workspace_size(B.LinearConfig(**sizes))


def test_linear_forward_does_not_compute_the_low_bits_rows():
    """2^32 + 8 rows (meta tensors: sizes without memory) are not 8 rows."""
    lc = B.LinearConfig(M=WRAP + 8, N=8, K=8)
    t = torch.empty(WRAP + 8, 8, dtype=torch.bfloat16, device="meta")
    w = torch.empty(8, 8, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="M: .* 32 bits"):
        B.moe_linear_forward(lc, t, w, t, torch.empty(1 << 20, dtype=torch.uint8, device="meta"))


@pytest.mark.parametrize("field", list(SIZES))
@pytest.mark.parametrize("sign", [1, -1])
def test_layer_config(field, sign):
    cfg = B.Config(**SIZES)
    assert B.validate_config(cfg) == B.MOE_OK
    bits = 64 if field == "capacity_rows" else 32
    wrong = SIZES[field] + sign * (1 << bits)
    with pytest.raises(ValueError, match=f"{field}: .* {bits} bits"):
        B.Config(**{**SIZES, field: wrong})
    with pytest.raises(ValueError, match=f"{field}: .* {bits} bits"):
        setattr(cfg, field, wrong)
    assert B.validate_config(cfg) == B.MOE_OK             # as it was
    assert B.validate_config(B.Config(**{**SIZES, "capacity_rows": 1 << 40})) == B.MOE_OK


def test_a_config_may_carry_other_attributes():
    cfg = B.Config(**SIZES)
    cfg.name = "a label"
    cfg.note = 1 << 80
    assert B.validate_config(cfg) == B.MOE_OK and cfg == B.Config(**SIZES)
