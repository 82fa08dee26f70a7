"""Calls around the experts on arrays of more than 2^31 elements, and of more blocks than a grid's first
dimension takes: the last rows are those of a call on them alone, bit for bit."""
import pytest
import torch

from block_cases import BF, F32, gen
from mixture_experts_layer_dispatch_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def big(g, shape, dtype=F32):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def route(logits, dw, ds, k, rc):
    T, E = logits.shape
    cfg = B.Config(T=T, H=128, I=128, E=E, k=k)
    sched = {"topk_idx": torch.full((T, k), -1, dtype=torch.int32, device="cuda"), "topk_w": torch.empty(T, k, device="cuda")}
    scores, dl, ws = torch.empty_like(logits), torch.empty_like(logits), B.alloc_error_word()
    B.moe_route_forward(cfg, rc, logits, sched, scores=scores)
    B.moe_route_backward(cfg, rc, logits, sched, dw, dl, ws, d_scores=ds)
    assert B.moe_check_device_error(ws) == 0
    return sched["topk_idx"], sched["topk_w"], scores, dl


@pytest.mark.parametrize("T,E,k", [((1 << 21) + 3, 1024, 4), ((1 << 24) + 3, 8, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route(T, E, k, score):
    g = gen(1)
    logits, dw, ds = big(g, (T, E)), big(g, (T, k)), big(g, (T, E))
    rc = B.RouteConfig(score=score, n_group=4, topk_group=2, group_top=2)
    whole = route(logits, dw, ds, k, rc)
    for rows in (slice(T - 1000, T), slice(T // 2, T // 2 + 1000)):
        part = route(logits[rows].clone(), dw[rows].clone(), ds[rows].clone(), k, rc)
        assert all(torch.equal(a[rows], b) for a, b in zip(whole, part))


@pytest.mark.parametrize("M,H", [((1 << 20) + 5, 8200), (140000, 16400)])
def test_norm(M, H):
    g = gen(2)
    x, dy = big(g, (M, H), BF), big(g, (M, H), BF)
    gamma = torch.rand(H, generator=g, device="cuda").to(BF) + 0.5

    def both(x, dy):
        nc = B.NormConfig(M=len(x), H=H)
        y, dx = torch.empty_like(x), torch.empty_like(x)
        mean, rstd = torch.empty(len(x), device="cuda"), torch.empty(len(x), device="cuda")
        dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(gamma)
        B.moe_norm_forward(nc, x, gamma, y, mean=mean, rstd=rstd)
        B.moe_norm_backward(nc, x, gamma, rstd, dy, dx, B.alloc_norm_workspace(nc), mean=mean, dgamma=dgamma, dbeta=dbeta)
        return y, mean, rstd, dx, dgamma, dbeta

    *whole, dgamma, dbeta = both(x, dy)
    for rows in (slice(M - 500, M), slice(M // 2, M // 2 + 500)):
        part = both(x[rows].clone(), dy[rows].clone())
        assert all(torch.equal(a[rows], b) for a, b in zip(whole, part))
    cols = torch.tensor([0, 1, 777, H // 2, H - 1], device="cuda")
    d = dy[:, cols].double()
    xh = (x[:, cols].double() - whole[1].double().unsqueeze(1)) * whole[2].double().unsqueeze(1)
    for got, t in ((dgamma, d * xh), (dbeta, d)):
        # sums of M / 256 values or fewer in a lane and 600 parts, in fp32; then bf16
        tol = (M / 256 + 600) * 2.0 ** -24 * t.abs().sum(0) + 2.0 ** -8 * t.sum(0).abs()
        assert ((got[cols].double() - t.sum(0)).abs() <= tol).all()


def test_w4_rows():
    g = gen(3)
    M, N, K = 1 << 20, 4096, 32
    x = big(g, (M, K), BF)
    wc = B.LinearW4Config(M=M, N=N, K=K, group=32, act="silu")
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.rand(1, N, generator=g, device="cuda").to(BF)

    def call(x):
        wc = B.LinearW4Config(M=len(x), N=N, K=K, group=32, act="silu")
        y = torch.empty(len(x), N, dtype=BF, device="cuda")
        B.moe_linear_w4_forward(wc, x, codes, scales, y, B.alloc_linear_w4_workspace(wc), residual=None)
        return y

    whole = call(x)
    assert whole.numel() > 1 << 31
    for rows in (slice(M - 1000, M), slice(M // 2, M // 2 + 1000)):
        assert torch.equal(whole[rows], call(x[rows].clone()))


@pytest.mark.parametrize("zeros", [False, True])
def test_w4_quantize(zeros):
    g = gen(4)
    E, N, K = 1024, 2048, 2176
    w = big(g, (E, N, K), BF)

    def call(w):
        wc = B.LinearW4Config(M=1, N=N, K=K, E=len(w), group=128)
        q = B.alloc_linear_w4_weights(wc, zeros)
        B.moe_linear_w4_quantize(wc, w, **q)
        return q

    whole = call(w)
    for e in (0, E // 2, E - 1):
        part = call(w[e:e + 1].clone())
        assert all(torch.equal(whole[n][e], part[n][0]) for n in part)
