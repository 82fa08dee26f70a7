"""A workspace that is another buffer of the same call is refused: it is written while the others are read
or written.  On the host, at the C entry points of routing with scores, norm and linear with 4-bit weights."""
import pytest

from mixture_experts_layer_dispatch_amd import binding as B
from test_around_refusals import ADDR, CALLS, call, no_gpu

WITH = ["moe_route_backward", "moe_schedule_from_topk", "moe_norm_backward", "moe_linear_w4_forward"]


@no_gpu
@pytest.mark.parametrize("name,arg", [(c, n) for c in WITH for n in CALLS[c]])
def test_refused(name, arg):
    assert call(name) == B.MOE_ERR_UNSUPPORTED_DEVICE
    assert call(name, ws=ADDR[arg]) == B.MOE_ERR_INVALID_ARG
