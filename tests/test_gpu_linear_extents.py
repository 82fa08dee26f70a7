"""linear at the ends of its sizes and values: the longest rows (N, K of 65536),
the most rows (2^24), matrices past 32-bit offsets, all rows in one of many
groups, subnormal values, and several macrobatches, each a call on its slice
of the rows."""
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


@pytest.mark.parametrize("counts", [None, [500000, 0, 548500]])
@pytest.mark.parametrize("N,K", [(2056, 72), (72, 2056)])
def test_rows_past_32_bit_offsets(N, K, counts):
    """More than 2^31 elements of y and dy, then of x and dx, in small whole numbers: every sum is exact in fp32."""
    M, step = 1048576, 1 << 17
    g = gen(8)
    E = len(counts) if counts else 0
    lead = (E,) if E else ()
    lc = B.LinearConfig(M=M, N=N, K=K, E=E)
    off = torch.tensor([0, 500000, 500000, 1048500], dtype=torch.int32, device="cuda") if E else None
    n = 1048500 if E else M
    x, dy = (torch.randint(-1, 2, (M, s), generator=g, device="cuda", dtype=torch.int8).to(BF) for s in (K, N))
    w = torch.randint(-2, 3, (*lead, N, K), generator=g, device="cuda").to(BF)
    ws = B.alloc_linear_workspace(lc)
    y, dx = torch.full_like(dy, -77.0), torch.full_like(x, -77.0)
    dw, db = torch.full_like(w, -77.0), torch.full((*lead, N), -77.0, dtype=BF, device="cuda")
    B.moe_linear_forward(lc, x, w, y, ws, offsets=off)
    B.moe_linear_backward(lc, x, w, None, dy, ws, dx=dx, dw=dw, db=db, offsets=off)
    assert B.moe_check_device_error(ws) == 0
    dw_ref, db_ref = torch.zeros(w.shape, device="cuda"), torch.zeros(db.shape, device="cuda")
    bounds = sorted({*range(0, n, step), n, *([500000] if E else [])})
    for a, b in zip(bounds, bounds[1:]):
        e = () if not E else (0 if b <= 500000 else 2,)
        xf, df, wf = x[a:b].float(), dy[a:b].float(), w[e].float()
        assert torch.equal(y[a:b], (xf @ wf.t()).to(BF)), a
        assert torch.equal(dx[a:b], (df @ wf).to(BF)), a
        dw_ref[e] += df.t() @ xf
        db_ref[e] += df.sum(0)
    assert torch.equal(dw, dw_ref.to(BF)) and torch.equal(db, db_ref.to(BF))
    assert (y[n:] == -77).all() and (dx[n:] == -77).all()


def _alone(E, e, n):
    return [n if i == e else 0 for i in range(E)]


@pytest.mark.parametrize("counts", [_alone(200, 0, 1500), _alone(200, 199, 1500), _alone(64, 31, 500),
                                    [1] * 300 + [1200] + [1] * 300, [2000] + [3] * 62, _alone(1024, 777, 3000)],
                         ids=["first", "last", "few", "middle", "hot", "thousand"])
@pytest.mark.parametrize("N,K", [(136, 200), (264, 2056)])
def test_most_rows_in_one_of_many_groups(N, K, counts):
    """The forms are chosen by the average group."""
    c = Lin(33, sum(counts) + 2, N, K, BF, "gelu", counts)
    out = c.outputs()
    c.run(out)
    c.check(out)


@pytest.mark.parametrize("M,counts", [(3, None), (40, None), (300, None), (4096, None), (90, [50, 0, 40])])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_subnormal_values(dtype, M, counts):
    """Operands below the type's smallest normal number count, and so do outputs there: whole multiples of
    the smallest subnormal number, so that every sum is exact."""
    N, K = 264, 2056
    unit = float(torch.finfo(dtype).smallest_normal) * torch.finfo(dtype).eps
    g = gen(9)
    E = len(counts) if counts else 0
    lead = (E,) if E else ()
    lc = B.LinearConfig(M=M, N=N, K=K, E=E, dtype=dtype)
    off = torch.tensor([0, 50, 50, 90], dtype=torch.int32, device="cuda") if E else None
    top = int(1 / torch.finfo(dtype).eps) // 2             # x and dy: up to half the smallest normal number
    ints = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g, device="cuda").double()  # noqa: E731
    xi, di, wi = ints(-top, top, M, K), ints(-top, top, M, N), ints(-1, 1, *lead, N, K)
    x, dy, w = (xi * unit).to(dtype), (di * unit).to(dtype), wi.to(dtype)
    assert torch.equal(x.double(), xi * unit)
    ws = B.alloc_linear_workspace(lc)
    y, dx, db = torch.full_like(dy, -77.0), torch.full_like(x, -77.0), torch.full((*lead, N), -77.0, dtype=dtype,
                                                                                 device="cuda")
    B.moe_linear_forward(lc, x, w, y, ws, offsets=off)
    B.moe_linear_backward(lc, None, w, None, dy, ws, dx=dx, db=db, offsets=off)
    for a, b, e in ([(0, M, ())] if not E else [(0, 50, (0,)), (50, 90, (2,))]):
        for got, want in ((y[a:b], xi[a:b] @ wi[e].t()), (dx[a:b], di[a:b] @ wi[e]), (db[e], di[a:b].sum(0))):
            assert want.abs().max() < 2 ** 24
            assert torch.equal(got, (want * unit).to(dtype))


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
