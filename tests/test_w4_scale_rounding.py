"""The 4-bit quantiser's scales are the quotients rounded once to the scales' type.  fp16 groups
whose quotient lies closer to a halfway number than fp32 tells apart: (hi - lo) / 15 = t - 2^-11 / 15
with t odd and above 2048, where fp16 has the even numbers."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_dispatch_amd import binding as B
from oracle import around

T = np.array([2063 + 16 * i for i in range(8)])


def groups(group):
    """[8, group] weights with hi = 15 t - 1 and lo = -(1 - 2^-11), both fp16 numbers."""
    w = np.zeros((8, group))
    w[:, 3], w[:, group - 5] = 15 * T - 1, -(1 - 2.0 ** -11)
    assert (w == w.astype(np.float16)).all()
    return w


@pytest.mark.parametrize("group", [32, 64, 128])
def test_oracle(group):
    _, scales, zeros = around.w4_quantize(groups(group), group, lambda a: a.astype(np.float16).astype(np.float64), True)
    np.testing.assert_array_equal(scales, (T - 1)[None])
    np.testing.assert_array_equal(zeros, np.zeros((1, 8)))


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
def test_kernel(group):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w = torch.tensor(groups(group), device="cuda").to(torch.float16)
    wc = B.LinearW4Config(M=1, N=8, K=group, group=group, dtype=torch.float16)
    q = B.alloc_linear_w4_weights(wc, True)
    B.moe_linear_w4_quantize(wc, w, **q)
    np.testing.assert_array_equal(q["scales"].double().cpu().numpy(), (T - 1)[None])
    codes, _, zeros = around.w4_quantize(w.double().cpu().numpy(), group,
                                         lambda a: a.astype(np.float16).astype(np.float64), True)
    np.testing.assert_array_equal(around.w4_codes(q["codes"].cpu().numpy()), codes)
    np.testing.assert_array_equal(q["zeros"].cpu().numpy(), zeros)


def test_rounding_to_odd_is_rounding_once():
    """Against whole-number arithmetic: quotients of whole numbers by 15, rounded half to even to 11 bits."""
    rng = np.random.default_rng(0)
    n = np.concatenate([rng.integers(1, 1 << 40, 2000), 15 * 2 * (2 * rng.integers(1024, 2048, 500) + 1) * (1 << 25) + 1,
                        15 * 2 * (2 * rng.integers(1024, 2048, 500) + 1) * (1 << 25)])
    got = around._to_odd(n / 15.0).astype(np.float64)
    for v, m in zip(got, n.tolist()):
        e = max(0, (m // 15).bit_length() - 11)             # 11 bits stay: q = m / (15 2^e)
        q, r = divmod(m, 15 << e)
        q += 2 * r > 15 << e or (2 * r == 15 << e and q % 2 == 1)
        f, b = divmod(v, 2.0 ** e)
        f += b > 2.0 ** e / 2 or (b == 2.0 ** e / 2 and f % 2 == 1)
        assert f == q, (m, v)
