"""The activations' tails on the GPU, to the relative precision that a 16-bit
output has there: x = 0 and bias = z make z exact, y = act(z) goes out rounded
once, and db of one row with dy = 1 is act'(z) rounded once.

Bounds, with e = 2^-24 (half a step of fp32), relative unless said:
  the normal distribution's fit  FIT = 7e-6: its approximation error of 6.5e-6 and
      the last roundings of 1 - q and of the exponential (8 e = 4.8e-7); the
      kernel takes it as 0 below z = -6, where it is at most 9.9e-10
  its density  (1.5 z^2 + 6) e: -z^2 / 2 has one rounding, its product with log2(e)
      and that constant's two more, each of z^2 / 2 e in the result; exp2 2 e,
      constants and products the rest
  sigmoid(v) = 1 / (1 + exp(-v)), p  ((2 |v| + 2) (1 - p) + 4) e: the product with
      log2(e) and that constant, exp2, weighted by exp(-v) / (1 + exp(-v)) = 1 - p;
      the addition and the reciprocal
  gelu_tanh's argument  7 e: four of the cubic term, the addition, the constant
      and its product, which moves the exponential by 7 |v| e
"""
import numpy as np
import pytest
import torch
from scipy.special import expit, ndtr

from block_cases import BF, FP, TINY, U, assert_within, n64
from mixture_experts_layer_dispatch_amd import binding as B

pytestmark = pytest.mark.gpu
IDS = {BF: "bf16", FP: "fp16"}
E, FIT = 2.0 ** -24, 7e-6
C, A = np.sqrt(2 / np.pi), 0.044715
REACH = {"gelu": 12.0, "gelu_tanh": 9.0, "silu": 80.0}     # (beyond: fp32 exponentials below the smallest normal number)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def reference(act, z):
    """act(z), act'(z) in 64 bits and the bounds of their fp32 errors."""
    if act == "gelu":
        cdf, pdf = ndtr(z), np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
        cerr = np.where(z < -6, cdf, FIT * cdf)
        y, yerr = z * cdf, np.abs(z) * cerr
        g, gerr = cdf + z * pdf, cerr + (1.5 * z * z + 6) * E * np.abs(z) * pdf + 2 * E * (cdf + np.abs(z) * pdf)
        return y, yerr + 2 * E * np.abs(y), g, gerr
    v, verr, slope = (z, 0, 1) if act == "silu" else (2 * C * (z + A * z ** 3), 7, 2 * C * (1 + 3 * A * z * z))
    p, q = expit(v), expit(-v)
    rel = (((2 + verr) * np.abs(v) + 2) * q + 4) * E
    qerr = p * rel + E                                       # of 1 - p, absolute
    y, yerr = z * p, np.abs(z) * p * (rel + 2 * E)
    zs = np.abs(z) * slope
    g, gerr = p + z * slope * p * q, p * rel + zs * p * (qerr + q * rel) + 10 * E * (p + zs * p * q)
    return y, yerr, g, gerr


def grid(dtype, reach):
    """Every value of the type from 2^-8 to `reach`, both signs, and 0; a multiple of 8 of them."""
    v = torch.arange(0, 1 << 15, dtype=torch.int32).to(torch.int16).view(dtype).double()
    v = v[(v >= 2.0 ** -8) & (v <= reach)]
    v = torch.cat([v, -v, torch.zeros(8)])
    return v[:v.numel() // 8 * 8].to(dtype).cuda()


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("act", list(REACH))
@pytest.mark.parametrize("M", [1, 200])                    # the streaming form's epilogue, the tiles'
def test_tails(M, act, dtype):
    z = grid(dtype, REACH[act])
    N = z.numel()
    lc = B.LinearConfig(M=M, N=N, K=8, dtype=dtype, act=act)
    ws = B.alloc_linear_workspace(lc)
    x, w = (torch.zeros(s, 8, dtype=dtype, device="cuda") for s in (M, N))
    y, zs = (torch.full((M, N), -77.0, dtype=dtype, device="cuda") for _ in range(2))
    B.moe_linear_forward(lc, x, w, y, ws, bias=z, z=zs)
    assert torch.equal(zs, z.expand(M, N))
    assert torch.equal(y, y[:1].expand(M, N))
    dy = torch.zeros(M, N, dtype=dtype, device="cuda")
    dy[0] = 1                                               # one row's derivative is the column's sum
    db = torch.full_like(z, -77.0)
    B.moe_linear_backward(lc, None, None, zs, dy, ws, db=db)
    want, werr, grad, gerr = reference(act, n64(z))
    u, tiny = U[dtype], TINY[dtype]
    assert_within("y", y[0], want, u * np.abs(want) + (1 + u) * werr + tiny)
    assert_within("act'", db, grad, u * np.abs(grad) + (1 + u) * gerr + tiny)
    if act == "gelu":
        assert np.max(np.abs(want[n64(z) < -6])) < 6e-9      # what the cut-off can leave out
