"""linear at the ends of its sizes: the longest rows (N, K of 65536), the most
rows (2^24), and several macrobatches, each a call on its slice of the rows."""
import pytest
import torch

from block_cases import BF, FP, gen, n64, randn, schedule
from mixture_experts_layer_dispatch_amd import binding as B
from test_gpu_linear import Lin, check_linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("M,counts", [(1, None), (40, None), (300, None), (45, [30, 0, 10]), (700, [300, 1, 399])])
@pytest.mark.parametrize("N,K,dtype", [(65536, 72, BF), (72, 65536, FP), (65536, 8, FP), (8, 65536, BF)])
def test_longest_rows(N, K, dtype, M, counts):
    c = Lin(M + N, M, N, K, dtype, "silu", counts)
    out = c.outputs()
    c.run(out)
    c.check(out)


def test_most_rows():
    """2^24 rows of small whole numbers: every sum is exact in fp32, in any order."""
    M, N, K = 1 << 24, 8, 16
    lc = B.LinearConfig(M=M, N=N, K=K, act="relu")
    g = gen(7)
    x, dy, z = (torch.randint(-1, 2, (M, n), generator=g, device="cuda").to(BF) for n in (K, N, N))
    w = torch.randint(-2, 3, (N, K), generator=g, device="cuda").to(BF)
    bias = torch.randint(-3, 4, (N,), generator=g, device="cuda").to(BF)
    ws = B.alloc_linear_workspace(lc)
    y, dx = torch.full_like(dy, -77.0), torch.full_like(x, -77.0)
    dw, db = torch.full_like(w, -77.0), torch.full_like(bias, -77.0)
    B.moe_linear_forward(lc, x, w, y, ws, bias=bias, residual=dy)
    B.moe_linear_backward(lc, x, w, z, dy, ws, dx=dx, dw=dw, db=db)
    dz = dy.double() * (z > 0)
    assert torch.equal(y.double(), (x.double() @ w.double().t() + bias.double()).clamp(min=0) + dy.double())
    assert torch.equal(dx.double(), dz @ w.double())
    assert torch.equal(dw, (dz.t() @ x.double()).to(BF))
    assert torch.equal(db, dz.sum(0).to(BF))
    assert B.moe_check_device_error(ws) == 0


@pytest.mark.parametrize("T,macrobatch,E,k,N", [(96, 32, 6, 3, 136), (60, 12, 90, 2, 72), (2048, 1024, 4, 2, 520)])
def test_macrobatches_one_by_one(T, macrobatch, E, k, N):
    """Macrobatch m: rows m * M * k onwards of the permuted rows, and the schedule's offsets[m]."""
    H = 128
    cfg, sched, ws = schedule(41, T, E, k, H, macrobatch)
    assert cfg.n_macro > 1
    Sm = macrobatch * k
    g = gen(42)
    x, w = randn(g, (T, H), BF), randn(g, (E, N, H), BF, H ** -0.5)
    bias, dy = randn(g, (E, N), BF), randn(g, (cfg.S, N), BF)
    lc = B.LinearConfig(M=Sm, N=N, K=H, E=E, act="gelu")
    lws = B.alloc_linear_workspace(lc)
    xs, dxs = (torch.full((cfg.S, H), -77.0, dtype=BF, device="cuda") for _ in range(2))
    y, z = (torch.full((cfg.S, N), -77.0, dtype=BF, device="cuda") for _ in range(2))
    dw, db = (torch.full((cfg.n_macro, *t.shape), -77.0, dtype=BF, device="cuda") for t in (w, bias))
    B.moe_permute_forward(cfg, sched, x, xs, ws)
    for m in range(cfg.n_macro):
        rows = slice(m * Sm, (m + 1) * Sm)
        off = sched["offsets"][m]
        B.moe_linear_forward(lc, xs[rows], w, y[rows], lws, bias=bias, z=z[rows], offsets=off)
        B.moe_linear_backward(lc, xs[rows], w, z[rows], dy[rows], lws, dx=dxs[rows], dw=dw[m], db=db[m], offsets=off)
    assert B.moe_check_device_error(ws) == 0 and B.moe_check_device_error(lws) == 0
    slot = sched["slot_of_row"].long()
    assert torch.equal(xs, x[slot // k])
    for m in range(cfg.n_macro):
        rows = slice(m * Sm, (m + 1) * Sm)
        off = sched["offsets"][m].tolist()
        assert off[0] == 0 and off[E] == Sm
        expert = sched["topk_idx"].view(-1)[slot[rows]].tolist()
        assert expert == [e for e in range(E) for _ in range(off[e + 1] - off[e])]
        out = {"y": y[rows], "z": z[rows], "dx": dxs[rows], "dw": dw[m], "db": db[m]}
        check_linear(out, xs[rows], w, bias, None, dy[rows], lc, off, Sm)
    o = randn(g, (cfg.S, H), BF)
    back = torch.full_like(x, -77.0)
    B.moe_permute_backward(cfg, sched, o, back, ws)
    row = sched["row_of_slot"].view(T, k).long()
    ref = sum(n64(o[row[:, j]]) for j in range(k))
    assert abs(n64(back) - ref).max() <= 2.0 ** -8 * abs(ref).max()
