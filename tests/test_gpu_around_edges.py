"""Calls around the experts that lie at an edge: weights that are all zero, reductions
that are split, calls on two streams at once, biases beyond the scores."""
import numpy as np
import pytest
import torch

from block_cases import U, assert_within, gen, n64, randn, sum_err
from mixture_experts_layer_dispatch_amd import binding as B
from oracle import around
from test_gpu_route import check as check_route

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("M", [1, 20, 64, 65, 150])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_weights_that_are_zero(M, group, dtype):
    """Codes of 8 without zeros.  fp16 takes the 8 off exactly; bf16 may take 8 times the sum of x off a
    sum of 8 x: two sums of at most `group` terms and one over the groups, of magnitudes of 16 |x| scale."""
    g = gen(M)
    N, K = 136, 384
    wc = B.LinearW4Config(M=M, N=N, K=K, group=group, dtype=dtype)
    x = randn(g, (M, K), dtype)
    codes = torch.full((N, K // 2), 0x88, dtype=torch.uint8, device="cuda")
    scales = torch.rand(K // group, N, generator=g, device="cuda").to(dtype)
    y = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    B.moe_linear_w4_forward(wc, x, codes, scales, y, B.alloc_linear_w4_workspace(wc))
    mag = 16 * np.abs(n64(x)).reshape(M, K // group, group).sum(2) @ np.abs(n64(scales))
    bound = sum_err(2 * group + K // group, mag) * (1 + 2 * U[dtype]) if dtype == BF else np.zeros_like(mag)
    assert_within("y", y, np.zeros((M, N)), bound)


@pytest.mark.parametrize("M,N,K,E,group,zeros", [(100, 1032, 4096, 0, 32, True), (300, 264, 8192, 0, 128, False),
                                                 (130, 72, 4096, 2, 64, False)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_split_reductions_on_two_streams_and_in_a_graph(M, N, K, E, group, zeros, dtype):
    """Few tiles and a long reduction; calls that overlap have a workspace each."""
    g = gen(M + N)
    wc = B.LinearW4Config(M=M, N=N, K=K, E=E, group=group, dtype=dtype)
    x = randn(g, (M, K), dtype)
    cs, ss = wc.shapes
    codes = torch.randint(0, 256, cs, generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(ss, generator=g, device="cuda") * K ** -0.5).to(dtype)
    z = torch.randint(0, 16, ss, generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    counts = [M - 37, 30] if E else None
    off = torch.tensor([0, M - 37, M - 7], dtype=torch.int32, device="cuda") if E else None
    wss = [B.alloc_linear_w4_workspace(wc) for _ in range(2)]
    ys = [torch.full((M, N), -3.0, dtype=dtype, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]

    def step(i):
        B.moe_linear_w4_forward(wc, x, codes, scales, ys[i], wss[i], zeros=z, offsets=off)

    torch.cuda.synchronize()
    for _ in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                step(i)
    torch.cuda.synchronize()
    rows = sum(counts) if E else M
    ref, _, mag = around.linear_w4(n64(x[:rows]), codes.cpu().numpy(), n64(scales), None if z is None else z.cpu().numpy(),
                                   offsets=None if off is None else off.tolist())
    u = U[dtype]
    tol = (sum_err(K + K // group + 2, mag) + u * np.abs(ref) + 2.0 ** -24) * (1 + 2 * u)
    for y in ys:
        assert_within("y", y[:rows], ref, tol)
        assert (y[rows:] == -3).all()
    assert torch.equal(ys[0], ys[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0)
    for _ in range(3):
        ys[0].fill_(-3)
        step(1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ys[0], ys[1])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,n_group,topk_group", [(40, 64, 6, 1, 1), (40, 512, 10, 8, 4), (20, 1023, 16, 33, 7)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_biases_beyond_the_scores(score, T, E, k, n_group, topk_group, group_top):
    """Biases so large that scores vanish beside them, a few infinite or NaN, and equal ones."""
    g = gen(E + k)
    inf = float("inf")
    logits = torch.randn(T, E, generator=g, device="cuda") * 2
    for bias in (torch.randint(-3, 4, (E,), generator=g, device="cuda").float() * 1e30,
                 torch.randint(-3, 4, (E,), generator=g, device="cuda").float() * 2.0 ** 20,
                 torch.full((E,), -0.25, device="cuda")):
        check_route(logits, k, bias, score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    bias[::7] = -inf
    bias[3::11] = float("nan")
    check_route(logits, k, bias, score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)
    bias[1::50] = inf
    check_route(logits, k, bias, score=score, n_group=n_group, topk_group=topk_group, group_top=1)
