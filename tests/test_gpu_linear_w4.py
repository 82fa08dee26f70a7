"""Linear with 4-bit weights on the GPU against the 64-bit reference, element by
element: the fp32 sum of K products of x with whole numbers (and a multiply-add
per group), then the epilogue's errors as for linear."""
import numpy as np
import pytest
import torch

from block_cases import (ACT_ERR, ACT_SLOPE, BF, FP, TINY, U, assert_within, gen, group_offsets, n64, randn, sum_err)
from mixture_experts_layer_dispatch_amd import binding as B
from oracle import around

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def weights(g, wc, zeros):
    """Random codes, scales of different sizes (some 0), zero points."""
    codes, groups = wc.shapes
    c = torch.randint(0, 256, codes, generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randn(groups, generator=g, device="cuda").exp_() * (0.3 * wc.K ** -0.5)
    s *= torch.rand(groups, generator=g, device="cuda") > 0.05
    z = torch.randint(0, 16, groups, generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return c, s.to(wc.dtype), z


def check(wc, zeros=True, bias=True, residual=True, counts=None, seed=0, in_place=False):
    g = gen(seed)
    M, N, K, E, dt = wc.M, wc.N, wc.K, wc.E, wc.dtype
    lead = (E,) if E else ()
    x = randn(g, (M, K), dt)
    codes, scales, z = weights(g, wc, zeros)
    b = randn(g, (*lead, N), dt, 0.5) if bias else None
    r = randn(g, (M, N), dt) if residual else None
    off = group_offsets(counts) if E else None
    ws = B.alloc_linear_w4_workspace(wc)
    y = torch.full((M, N), float("nan"), dtype=dt, device="cuda")
    a = dict(zeros=z, bias=b, offsets=off)
    B.moe_linear_w4_forward(wc, x, codes, scales, y, ws, residual=r, **a)
    assert B.moe_check_device_error(ws) == 0
    rows = sum(counts) if E else M
    assert torch.isnan(y[rows:]).all()                       # rows in no group are left as they were
    ref, lin, mag = around.linear_w4(n64(x[:rows]), codes.cpu().numpy(), n64(scales),
                                     None if z is None else z.cpu().numpy(), n64(b),
                                     None if r is None else n64(r[:rows]), wc.act, None if off is None else off.tolist())
    u, res = U[dt], 0.0 if r is None else np.abs(n64(r[:rows]))
    tol = ACT_SLOPE * sum_err(K + K // wc.group + 2, mag) + ACT_ERR * np.maximum(np.abs(lin), 1) * (wc.act != "none")
    tol = tol + sum_err(0, np.abs(ref) + res)
    assert_within("y", y[:rows], ref, (tol + u * np.abs(ref) + TINY[dt]) * (1 + 2 * u))
    # again into the residual itself: the same bits
    if residual:
        y2 = r.clone()
        B.moe_linear_w4_forward(wc, x, codes, scales, y2, ws, residual=y2, **a)
        assert torch.equal(y2[:rows], y[:rows])


DENSE = [  # M, N, K, group
    (1, 8, 32, 32), (1, 4096, 4096, 128), (3, 24, 64, 64), (4, 1000, 96, 32), (7, 136, 320, 64), (15, 128, 128, 128),
    (16, 16, 384, 128), (17, 264, 1056, 32), (31, 72, 1088, 64), (33, 520, 640, 128), (48, 128, 256, 32),
    (64, 136, 512, 128), (65, 200, 192, 64), (100, 1032, 2080, 32), (127, 128, 448, 64), (129, 264, 384, 128),
    (200, 96, 96, 32), (257, 392, 256, 128), (300, 520, 1120, 32), (513, 256, 576, 64), (1000, 136, 128, 32)]


@pytest.mark.parametrize("M,N,K,group", DENSE)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("zeros", [False, True])
def test_dense(M, N, K, group, dtype, zeros):
    check(B.LinearW4Config(M=M, N=N, K=K, group=group, dtype=dtype), zeros, bias=M % 2 == 0, residual=M % 3 == 0,
          seed=M)


@pytest.mark.parametrize("act", list(B.ACTS))
@pytest.mark.parametrize("M", [2, 40, 150])
def test_activations(act, M):
    check(B.LinearW4Config(M=M, N=136, K=256, group=64, act=act), seed=M)


GROUPED = [  # counts, rows behind them, N, K, group
    ([1], 0, 16, 32, 32), ([0, 3, 0], 2, 136, 128, 64), ([5, 0, 0, 17, 1, 16, 33], 3, 72, 320, 64),
    ([1] * 70, 0, 40, 256, 128), ([0] * 69 + [200], 5, 128, 192, 32), ([2, 0, 3] * 60, 1, 264, 128, 128),
    ([64, 65, 63, 128, 129, 0, 1], 0, 200, 160, 32), ([300, 0, 20], 7, 136, 256, 64), ([40] * 30, 0, 136, 384, 128),
    ([0, 0, 0], 4, 16, 64, 32), ([700], 1, 24, 64, 64), ([130] * 9, 0, 392, 128, 32)]


@pytest.mark.parametrize("counts,rest,N,K,group", GROUPED)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_grouped(counts, rest, N, K, group, dtype):
    wc = B.LinearW4Config(M=sum(counts) + rest, N=N, K=K, E=len(counts), group=group, dtype=dtype, act="silu")
    check(wc, zeros=len(counts) % 2 == 1, counts=counts, seed=N, residual=rest % 2 == 0)


def test_many_experts():
    rng = np.random.default_rng(4)
    counts = rng.poisson(0.4, 1024).tolist()
    check(B.LinearW4Config(M=sum(counts), N=64, K=256, E=1024, group=128), zeros=False, counts=counts, residual=False)
    counts = rng.poisson(20, 100).tolist()
    check(B.LinearW4Config(M=sum(counts), N=136, K=128, E=100, group=64), counts=counts, residual=False)


@pytest.mark.parametrize("M,E", [(5, 0), (100, 0), (300, 0), (30, 3), (200, 3)])
def test_whole_numbers_exactly(M, E):
    """x and weights of whole numbers: every product and sum is exact, so y is, too."""
    g = gen(21)
    N, K, group = 136, 256, 32
    wc = B.LinearW4Config(M=M, N=N, K=K, E=E, group=group, dtype=FP)
    codes, _, z = weights(g, wc, True)
    scales = (2.0 ** torch.randint(0, 2, wc.shapes[1], generator=g, device="cuda")).to(FP)
    x = torch.randint(-1, 2, (M, K), generator=g, device="cuda").to(FP)
    off = group_offsets([M // 3] * 3) if E else None
    y = torch.empty(M, N, dtype=FP, device="cuda")
    ws = B.alloc_linear_w4_workspace(wc)
    for zz in (None, z):
        B.moe_linear_w4_forward(wc, x, codes, scales, y, ws, zeros=zz, offsets=off)
        ref, _, mag = around.linear_w4(n64(x), codes.cpu().numpy(), n64(scales), None if zz is None else zz.cpu().numpy(),
                                       offsets=None if off is None else off.tolist())
        assert mag.max() < 2 ** 24
        rows = M // 3 * 3 if E else M                        # (the others are in no group)
        assert torch.equal(y[:rows], torch.tensor(ref, device="cuda").to(FP)[:rows])


@pytest.mark.parametrize("M", [3, 90, 200])
def test_infinite_and_missing_values_stay_in_their_row(M):
    g = gen(22)
    wc = B.LinearW4Config(M=M, N=72, K=256, group=64)
    x = randn(g, (M, 256), BF)
    codes, scales, z = weights(g, wc, True)
    ws, good, bad = B.alloc_linear_w4_workspace(wc), *(torch.empty(M, 72, dtype=BF, device="cuda") for _ in range(2))
    B.moe_linear_w4_forward(wc, x, codes, scales, good, ws, zeros=z)
    x[1, 33], x[2, 255] = float("inf"), float("nan")
    B.moe_linear_w4_forward(wc, x, codes, scales, bad, ws, zeros=z)
    rest = [i for i in range(M) if i not in (1, 2)]
    assert torch.equal(good[rest], bad[rest])
    assert bad[2].isnan().all() and not bad[1].isfinite().any()


def test_offsets_that_descend_or_leave_the_rows():
    g = gen(23)
    for M, big in ((40, 50), (400, 500)):
        wc = B.LinearW4Config(M=M, N=136, K=128, E=4, group=128)
        x = randn(g, (M, 128), BF)
        codes, scales, _ = weights(g, wc, False)
        ws = B.alloc_linear_w4_workspace(wc)
        guard = torch.full((M + 64, 136), 5.0, dtype=BF, device="cuda")
        y = guard[32:32 + M]
        for off in ([0, M // 2, M // 4, M, M], [0, 10, 20, 30, big], [-5, 10, 20, 30, M], [0, M, 0, M, 0]):
            o = torch.tensor(off, dtype=torch.int32, device="cuda")
            B.moe_linear_w4_forward(wc, x, codes, scales, y, ws, offsets=o)
            assert B.moe_check_device_error(ws) == B.DEVERR_BAD_OFFSETS
            assert torch.all(guard[:32] == 5) and torch.all(guard[32 + M:] == 5)


def test_a_weight_past_32_bit_offsets():
    """Codes of more than 2^32 weights and 2^31 bytes: the last experts' products."""
    E, N, K = 1024, 2048, 2176
    wc = B.LinearW4Config(M=64, N=N, K=K, E=E, group=128)
    g = gen(24)
    codes, scales, _ = weights(g, wc, False)
    assert codes.numel() > 1 << 31
    x = randn(g, (64, K), BF)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E - 1], off[E] = 30, 64
    off[1:E - 1] = 2
    y, ws = torch.empty(64, N, dtype=BF, device="cuda"), B.alloc_linear_w4_workspace(wc)
    B.moe_linear_w4_forward(wc, x, codes, scales, y, ws, offsets=off)
    for e, r in ((0, slice(0, 2)), (E - 2, slice(2, 30)), (E - 1, slice(30, 64))):
        ref, _, mag = around.linear_w4(n64(x[r]), codes[e].cpu().numpy(), n64(scales[e]))
        assert_within(f"expert {e}", y[r], ref, (sum_err(K + 20, mag) + U[BF] * np.abs(ref)) * (1 + 2 * U[BF]))


@pytest.mark.parametrize("M,N", [(1 << 24, 8), (40000, 2056)])
def test_many_rows(M, N):
    wc = B.LinearW4Config(M=M, N=N, K=32, group=32)
    g = gen(25)
    x = torch.randn(M, 32, generator=g, device="cuda", dtype=BF)
    codes, scales, z = weights(g, wc, True)
    y, ws = torch.full((M, N), float("nan"), dtype=BF, device="cuda"), B.alloc_linear_w4_workspace(wc)
    B.moe_linear_w4_forward(wc, x, codes, scales, y, ws, zeros=z)
    w = torch.tensor(around.w4_weights(codes.cpu().numpy(), n64(scales), z.cpu().numpy()), device="cuda")
    for a in range(0, M, 1 << 20):
        ref = x[a:a + (1 << 20)].double() @ w.t()
        mag = x[a:a + (1 << 20)].double().abs() @ w.abs().t()
        err = (y[a:a + (1 << 20)].double() - ref).abs()
        assert (err <= (sum_err(36, mag) + U[BF] * ref.abs()) * (1 + 2 * U[BF])).all()


@pytest.mark.parametrize("M,E", [(3, 0), (200, 0), (50, 5), (600, 5)])
def test_graph_and_stream(M, E):
    g = gen(26)
    N, K = 136, 256
    wc = B.LinearW4Config(M=M, N=N, K=K, E=E, group=128, act="gelu")
    x = randn(g, (M, K), BF)
    codes, scales, _ = weights(g, wc, False)
    off = group_offsets([M // 5] * 5) if E else None
    ws, y = B.alloc_linear_w4_workspace(wc), torch.empty(M, N, dtype=BF, device="cuda")

    def step():
        B.moe_linear_w4_forward(wc, x, codes, scales, y, ws, offsets=off)

    step()
    first = y.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        y.fill_(-3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, first)
    side = torch.cuda.Stream()
    y.fill_(-3)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    assert torch.equal(y, first)


# ------------------------------------------------------------------ quantiser
@pytest.mark.parametrize("shape", [(8, 32), (24, 96), (136, 1152), (3, 16, 640), (5, 40, 512)])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize(shape, dtype, group, zeros):
    *lead, N, K = shape
    K = (K + group - 1) // group * group
    g = gen(27)
    w = randn(g, (*lead, N, K), dtype, K ** -0.5)
    w[..., 1, :group] = 0
    w[..., 2, :group] = w[..., 2, :group].abs()
    w[..., 3, :] = torch.randint(-7, 8, (K,), generator=g, device="cuda").to(dtype) / 2          # ties
    w[..., 4, :group] = torch.finfo(dtype).max
    w[..., 5, :group] = torch.finfo(dtype).smallest_normal
    wc = B.LinearW4Config(M=1, N=N, K=K, E=lead[0] if lead else 0, group=group, dtype=dtype)
    q = B.alloc_linear_w4_weights(wc, zeros)
    for t in q.values():
        t.fill_(1)
    B.moe_linear_w4_quantize(wc, w, **q)
    codes, scales, z = around.w4_quantize(n64(w), group, lambda a: n64(torch.from_numpy(a).to(dtype)), zeros)
    np.testing.assert_array_equal(n64(q["scales"]), scales)
    np.testing.assert_array_equal(around.w4_codes(q["codes"].cpu().numpy()), codes)
    if zeros:
        np.testing.assert_array_equal(q["zeros"].cpu().numpy(), z)


def test_quantised_product_is_near_the_weights():
    """The quantiser's weights in the product: half a step of a group's scale per weight."""
    g = gen(28)
    M, N, K = 33, 128, 512
    w = randn(g, (N, K), BF, K ** -0.5)
    wc = B.LinearW4Config(M=M, N=N, K=K, group=64)
    q = B.alloc_linear_w4_weights(wc)
    B.moe_linear_w4_quantize(wc, w, **q)
    x, y = randn(g, (M, K), BF), torch.empty(M, N, dtype=BF, device="cuda")
    B.moe_linear_w4_forward(wc, x, q["codes"], q["scales"], y, B.alloc_linear_w4_workspace(wc))
    half = np.repeat(n64(q["scales"]).T, 64, 1) * (0.5 + 8 * U[BF])
    ref = n64(x) @ n64(w).T
    assert_within("y", y, ref, np.abs(n64(x)) @ half.T + U[BF] * np.abs(ref) * 2 + 1e-3)
