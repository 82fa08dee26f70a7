"""GPU parity of the linear operator (dense and grouped by expert) against the
64-bit reference, forward and backward: every activation and type, one row to
many, sizes that fill no tile, empty and one-row groups, rows in no group,
weights past 32-bit offsets, bad offsets, other streams, captured graphs."""
import numpy as np
import pytest
import torch

from block_cases import (ACT_ERR, ACT_SLOPE, BF, FP, TINY, U, assert_within, gen, group_offsets, n64, randn, sum_err)
from mixture_experts_layer_dispatch_amd import binding as B
from oracle import blocks

pytestmark = pytest.mark.gpu
IDS = {BF: "bf16", FP: "fp16"}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Lin:
    def __init__(self, seed, M, N, K, dtype=BF, act="none", counts=None, bias=True, residual=True):
        """counts: the groups' sizes (their sum may be below M: the rows behind are in no group)."""
        g = gen(seed)
        E = 0 if counts is None else len(counts)
        lead = (E,) if E else ()
        self.lc = B.LinearConfig(M=M, N=N, K=K, E=E, dtype=dtype, act=act)
        self.x, self.w = randn(g, (M, K), dtype), randn(g, (*lead, N, K), dtype, K ** -0.5)
        self.bias = randn(g, (*lead, N), dtype) if bias else None
        self.res = randn(g, (M, N), dtype) if residual else None
        self.dy = randn(g, (M, N), dtype)
        self.off = None if counts is None else group_offsets(counts)
        self.off_list = None if counts is None else self.off.tolist()
        self.live = M if counts is None else sum(counts)
        self.ws = B.alloc_linear_workspace(self.lc)

    def outputs(self, fill=-77.0):
        lc, dt = self.lc, self.lc.dtype
        full = lambda like: torch.full(like, fill, dtype=dt, device="cuda")  # noqa: E731
        return {"y": full((lc.M, lc.N)), "z": full((lc.M, lc.N)), "dx": full((lc.M, lc.K)),
                "dw": full(tuple(self.w.shape)), "db": full((*self.w.shape[:-1],))}

    def run(self, out, stream=None):
        B.moe_linear_forward(self.lc, self.x, self.w, out["y"], self.ws, bias=self.bias, residual=self.res,
                             z=out["z"], offsets=self.off, stream=stream)
        B.moe_linear_backward(self.lc, self.x, self.w, out["z"], self.dy, self.ws, dx=out["dx"], dw=out["dw"],
                              db=out["db"], offsets=self.off, stream=stream)

    def check(self, out, untouched=-77.0):
        n = self.live
        check_linear(out, self.x, self.w, self.bias, self.res, self.dy, self.lc, self.off_list, n)
        for name in ("y", "z", "dx"):
            assert (out[name][n:] == untouched).all(), f"{name}: rows in no group were written"
        assert B.moe_check_device_error(self.ws) == 0


def check_linear(out, x, w, b, r, dy, lc, off, n):
    """Forward and backward outputs of the first n rows against the 64-bit reference."""
    dt, act = lc.dtype, lc.act
    u, tiny = U[dt], TINY[dt]
    x, w, b, r, dy = (n64(t) for t in (x, w, b, r, dy))
    y, z, mag = blocks.linear(x, w, b, r, act, off)
    zerr = sum_err(lc.K + 2, mag)
    assert_within("z", out["z"][:n], z[:n], (u * np.abs(z) + zerr + tiny)[:n])
    yerr = ACT_SLOPE * zerr + ACT_ERR * np.maximum(np.abs(z), 1) if act != "none" else zerr
    big = np.abs(y) + (np.abs(r) if r is not None else 0)
    assert_within("y", out["y"][:n], y[:n], (u * np.abs(y) + (1 + u) * yerr + 2.0 ** -23 * big + tiny)[:n])
    # the backward reads the stored z
    check_products(out, x, w, n64(out["z"]), dy, lc, off, n)


def check_products(out, x, w, zs, dy, lc, off, n):
    """Those of dx, dw and db that are in `out`, for the stored z."""
    dt, act = lc.dtype, lc.act
    u, tiny = U[dt], TINY[dt]
    x, w, zs, dy = (n64(t) if isinstance(t, torch.Tensor) else t for t in (x, w, zs, dy))
    if not {"dx", "dw", "db"} & set(out):
        return
    ref = blocks.linear_backward(x, w, zs, dy, act, off)
    # dz: rounded once to the type (exact for act "none"), and fp32 errors of act'
    rel = u if act != "none" else 0.0
    gerr = np.abs(dy) * (ACT_ERR * np.maximum(np.abs(zs), 1) if act != "none" else 0) + tiny
    one = blocks.linear_backward(np.abs(x), np.abs(w), zs, gerr, "none", off)
    for name, red in (("dx", lc.N), ("dw", lc.M), ("db", lc.M)):
        if out.get(name) is None:
            continue
        want, m = ref[name], ref["mag"][name]
        tol = u * np.abs(want) + (1 + u) * ((rel if name != "db" else 0) * m + one[name] + sum_err(red, m)) + tiny
        got = out[name]
        if name == "dx":
            got, want, tol = got[:n], want[:n], tol[:n]
        assert_within(name, got, want, tol)


DENSE = [(1, 8, 8), (1, 4096, 1024), (3, 264, 136), (48, 200, 2056), (64, 1544, 72), (130, 1608, 2104), (16, 128, 64), (17, 1000, 520), (64, 72, 8), (65, 136, 200),
         (129, 384, 328), (300, 1032, 256), (777, 520, 1544), (1024, 512, 768), (1300, 2056, 264)]


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense_sizes(M, N, K, dtype):
    c = Lin(M + N + K, M, N, K, dtype, "silu")
    out = c.outputs()
    c.run(out)
    c.check(out)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("act", list(B.ACTS))
@pytest.mark.parametrize("bias,residual", [(True, True), (False, False)])
@pytest.mark.parametrize("M", [5, 200])
def test_activations_biases_residuals(M, act, bias, residual, dtype):
    c = Lin(91, M, 136, 192, dtype, act, None, bias, residual)
    out = c.outputs()
    c.run(out)
    c.check(out)


COUNTS = [[150, 130, 170, 0, 200], [100, 90, 70], [0, 0, 0], [1], [0, 1, 0, 5, 64], [65, 0, 63, 128, 1], [300, 7, 0, 520], [3] * 70, [40] * 33,
          [1000, 0, 0, 2], [257, 256, 255, 511, 513]]


@pytest.mark.parametrize("behind", [0, 9])
@pytest.mark.parametrize("counts", COUNTS, ids=[f"groups{i}" for i in range(len(COUNTS))])
@pytest.mark.parametrize("N,K,dtype", [(136, 200, BF), (512, 256, BF), (264, 320, FP)])
def test_groups(counts, behind, N, K, dtype):
    c = Lin(17, sum(counts) + behind or 1, N, K, dtype, "gelu_tanh", counts)
    out = c.outputs()
    c.run(out)
    c.check(out)
    again = c.outputs()
    c.run(again)
    for n in out:
        assert torch.equal(out[n], again[n]), n


def test_many_experts():
    rng = np.random.default_rng(5)
    c = Lin(18, 700, 64, 72, BF, "relu", list(np.bincount(rng.integers(0, 1024, 700), minlength=1024)))
    out = c.outputs()
    c.run(out)
    c.check(out)


# sizes whose products have enough 256 x 256 tiles to take them, with reduction
# lengths of no, one and several 64-deep steps and remainders of all kinds
@pytest.mark.parametrize("K", [8, 64, 72, 128, 192, 200, 256, 328, 520])
def test_large_dense_forward(K):
    c = Lin(19, 4100, 2056, K, BF if K % 16 else FP, "gelu")
    out = c.outputs()
    for _ in range(3):
        B.moe_linear_forward(c.lc, c.x, c.w, out["y"], c.ws, bias=c.bias, residual=c.res, z=out["z"])
        check_linear({"y": out["y"], "z": out["z"]}, c.x, c.w, c.bias, c.res, c.dy, c.lc, None, 4100)
        out = c.outputs()


@pytest.mark.parametrize("N", [8, 64, 72, 128, 192, 200, 256, 328, 520])
def test_large_dense_input_gradient(N):
    c = Lin(29, 4100, N, 2056, BF if N % 16 else FP, "none")
    dx = torch.full_like(c.x, -77.0)
    B.moe_linear_backward(c.lc, None, c.w, None, c.dy, c.ws, dx=dx)
    check_products({"dx": dx}, c.x, c.w, c.dy, c.dy, c.lc, None, 4100)


@pytest.mark.parametrize("M", [256, 264, 300, 321, 383, 448, 577])
def test_large_dense_weight_gradient(M):
    c = Lin(39, M, 2056, 4104, BF if M % 2 else FP, "relu")
    dw = torch.full_like(c.w, -77.0)
    z = randn(gen(5), (M, 2056), c.lc.dtype)
    B.moe_linear_backward(c.lc, c.x, None, z, c.dy, c.ws, dw=dw)
    check_products({"dw": dw}, c.x, c.w, z, c.dy, c.lc, None, M)


@pytest.mark.parametrize("counts", [[900, 0, 1100, 500], [257, 256, 255, 511, 513], [1300, 1, 64, 0, 700]])
def test_large_groups(counts):
    c = Lin(49, sum(counts) + 3, 1032, 2056, BF, "silu", counts)
    out = c.outputs()
    c.run(out)
    c.check(out)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("act", list(B.ACTS))
def test_activations_at_the_ends_of_the_type(act, dtype):
    """Pre-activations up to the type's largest and lowest values (a mask's fill, an outlier)."""
    f = torch.finfo(dtype)
    z = torch.tensor([f.min, f.min / 2, -1e4, -30, -8, -6.1, -5.9, -1e-3, 0.0, 1e-3, 5.9, 6.1, 8, 30, 1e4, f.max],
                     dtype=torch.float64).to(dtype).cuda()
    lc = B.LinearConfig(M=8, N=16, K=8, dtype=dtype, act=act)
    x, w = torch.zeros(8, 8, dtype=dtype, device="cuda"), torch.zeros(16, 8, dtype=dtype, device="cuda")
    out = {"y": torch.empty(8, 16, dtype=dtype, device="cuda"), "z": torch.empty(8, 16, dtype=dtype, device="cuda")}
    ws = B.alloc_linear_workspace(lc)
    B.moe_linear_forward(lc, x, w, out["y"], ws, bias=z, z=out["z"])
    dy = torch.ones(8, 16, dtype=dtype, device="cuda")
    out.update(dx=torch.empty_like(x), dw=torch.empty_like(w), db=torch.empty_like(z))
    B.moe_linear_backward(lc, x, w, out["z"], dy, ws, dx=out["dx"], dw=out["dw"], db=out["db"])
    assert torch.equal(out["z"], z.expand(8, 16))
    with np.errstate(over="ignore"):
        check_linear(out, x, w, z, None, dy, lc, None, 8)


# groups whose products have enough 256 x 256 tiles: of x W^T, then of dz W and dW
@pytest.mark.parametrize("counts", [[900, 0, 1100, 600], [1257, 1256, 255, 1, 513], [1300, 1, 64, 0, 1700]])
@pytest.mark.parametrize("N,K", [(4104, 328), (328, 4104)])
def test_large_groups_of_many_tiles(N, K, counts):
    c = Lin(69, sum(counts) + 3, N, K, FP, "relu", counts)
    out = c.outputs()
    c.run(out)
    c.check(out)


@pytest.mark.parametrize("M", [512, 520, 575, 577, 639, 704])
def test_large_dense_weight_gradient_of_more_rows(M):
    c = Lin(79, M, 2056, 4104, FP if M % 2 else BF, "relu")
    dw = torch.full_like(c.w, -77.0)
    z = randn(gen(5), (M, 2056), c.lc.dtype)
    B.moe_linear_backward(c.lc, c.x, None, z, c.dy, c.ws, dw=dw)
    check_products({"dw": dw}, c.x, c.w, z, c.dy, c.lc, None, M)


# one round of 256 x 256 tiles and some left over, of x W^T, then of dz W; of dW
@pytest.mark.parametrize("M,counts", [(4200, None), (4700, None), (3700, [1700, 1, 64, 0, 1900]),
                                      (4500, [300, 2000, 130, 2000, 5, 60])])
@pytest.mark.parametrize("N,K,dtype", [(4232, 136, BF), (136, 4232, FP)])
def test_tiles_behind_the_last_whole_round(M, counts, N, K, dtype):
    c = Lin(99, M, N, K, dtype, "gelu", counts)
    out = c.outputs()
    c.run(out)
    c.check(out)


@pytest.mark.parametrize("M,counts", [(600, None), (1300, [513, 787])])
def test_weight_tiles_behind_the_last_whole_round(M, counts):
    c = Lin(109, M, 2184, 8200 if counts is None else 4232, BF, "silu", counts)
    dw = torch.full_like(c.w, -77.0)
    z = randn(gen(5), (M, 2184), c.lc.dtype)
    B.moe_linear_backward(c.lc, c.x, None, z, c.dy, c.ws, dw=dw, offsets=c.off)
    check_products({"dw": dw}, c.x, c.w, z, c.dy, c.lc, c.off_list, M)


# few tiles and long reductions: several parts each, forward and (N long) for dx
@pytest.mark.parametrize("counts", [[60, 0, 140], [0, 0, 1], [33, 5, 0, 64, 1], [200, 129, 300], [16] * 3])
@pytest.mark.parametrize("N,K", [(264, 2056), (1800, 136), (1640, 1544)])
def test_split_reductions_of_groups(N, K, counts):
    c = Lin(89, sum(counts) + 5, N, K, BF if N == 264 else FP, "gelu", counts)
    out = c.outputs()
    c.run(out)
    c.check(out)
    again = c.outputs()
    c.run(again)
    for n in out:
        assert torch.equal(out[n], again[n]), n


def test_outputs_stored_past_the_caches():
    """Outputs of more than 32 MB, and lists of tiles for few groups."""
    c = Lin(59, 4100, 4104, 72, BF, "relu")
    out = c.outputs()
    c.run(out)
    c.check(out)
    c = Lin(60, 4100, 72, 4104, FP, "silu")               # dx, with db in front of its tiles
    out = c.outputs()
    c.run(out)
    c.check(out)
    rng = np.random.default_rng(6)
    c = Lin(61, 17000, 1032, 64, BF, "silu", list(np.bincount(rng.integers(0, 110, 16990), minlength=110)))
    out = c.outputs()
    c.run(out)
    c.check(out)
    c = Lin(62, 20000, 2048, 64, BF, "relu", [9000, 0, 3001, 7990])
    out = c.outputs()
    c.run(out)
    c.check(out)


def test_groups_may_start_behind_the_first_row():
    c = Lin(63, 300, 136, 72, BF, "gelu", [100, 0, 150])
    out = c.outputs()
    c.run(out)
    pad = torch.full_like(c.x[:7], float("nan"))
    for name, fill in (("x", pad), ("res", c.res[:7]), ("dy", c.dy[:7] * float("nan"))):
        setattr(c, name, torch.cat([fill, getattr(c, name)])[:300].contiguous())
    c.off = c.off + 7
    got = c.outputs()
    c.run(got)
    for n in ("y", "z", "dx"):
        assert torch.equal(got[n][7:257], out[n][:250]), n
        assert (got[n][:7] == -77).all() and (got[n][257:] == -77).all(), n
    for n in ("dw", "db"):
        assert torch.equal(got[n], out[n]), n


def test_residual_may_be_the_output():
    for M in (3, 300):
        c = Lin(20, M, 264, 136, BF, "relu")
        out = c.outputs()
        c.run(out)
        y = c.res.clone()
        B.moe_linear_forward(c.lc, c.x, c.w, y, c.ws, bias=c.bias, residual=y)
        assert torch.equal(y, out["y"])


@pytest.mark.parametrize("counts", [None, [60, 0, 140]])
def test_each_gradient_alone(counts):
    c = Lin(21, 200, 136, 72, BF, "silu", counts)
    out = c.outputs()
    c.run(out)
    for name in ("dx", "dw", "db"):
        one = c.outputs()
        B.moe_linear_backward(c.lc, c.x if name == "dw" else None, c.w if name == "dx" else None, out["z"], c.dy, c.ws,
                              offsets=c.off, **{name: one[name]})
        assert torch.equal(one[name], out[name]), name


def test_rows_and_experts_do_not_mix():
    """Infinities and NaN stay in their row (or expert); rows in no group are not read."""
    counts = [30, 0, 50, 20]
    c = Lin(22, 110, 72, 136, BF, "none", counts, residual=False)
    out = c.outputs()
    c.run(out)
    nan, inf = float("nan"), float("inf")
    c.x[35] = inf
    c.x[100:] = nan                                       # behind the last group
    c.dy[100:] = nan
    c.w[3, 5, 6] = nan
    got = c.outputs()
    c.run(got)
    rows = [r for r in range(100) if r != 35]
    for n in ("y", "z"):
        cols = [j for j in range(72) if j != 5]
        assert torch.equal(got[n][rows][:, cols], out[n][rows][:, cols]), n
        assert torch.equal(got[n][:80][[r for r in rows if r < 80]], out[n][:80][[r for r in rows if r < 80]]), n
        assert torch.isnan(got[n][80:100, 5]).all() and not torch.isfinite(got[n][35]).any()
    assert torch.equal(got["dx"][:80], out["dx"][:80])
    for n in ("dw", "db"):
        assert torch.equal(got[n][0], out[n][0]) and torch.equal(got[n][3], out[n][3]), n
        assert (got[n][1] == 0).all(), n
    assert torch.equal(got["db"], out["db"])
    assert (got["y"][100:] == -77).all() and (got["dx"][100:] == -77).all()


@pytest.mark.parametrize("N,K,counts", [(4232, 136, [1700, 1, 64, 0, 1900]), (136, 4232, [1700, 1, 64, 0, 1900]),
                                        (2184, 4232, [787, 513]), (264, 2056, [60, 0, 140])])
def test_large_tiles_and_split_reductions_keep_groups_apart(N, K, counts):
    """NaN in the last group and behind it, in every operand: the groups before it stay as they were."""
    c = Lin(25, sum(counts) + 21, N, K, BF, "none", counts)
    out = c.outputs()
    c.run(out)
    n, nan = sum(counts[:-1]), float("nan")
    for name in ("x", "dy", "res"):
        getattr(c, name)[n:] = nan
    c.w[-1] = nan
    c.bias[-1] = nan
    got = c.outputs()
    c.run(got)
    for name in ("y", "z", "dx"):
        assert torch.equal(got[name][:n], out[name][:n]), name
        assert (got[name][c.live:] == -77).all(), name
    for name in ("dw", "db"):
        assert torch.equal(got[name][:-1], out[name][:-1]), name
        assert torch.isnan(got[name][-1]).all(), name


@pytest.mark.parametrize("E", [7, 90])
def test_overlapping_groups_stay_inside_the_workspace(E):
    """Offsets that go back and forth: more tiles than any valid offsets have."""
    M, N, K = 200, 136, 72
    c = Lin(24, M, N, K, BF, "silu", [M] + [0] * (E - 1))
    c.off = torch.tensor([0, M] * ((E + 1) // 2) + [0] * ((E + 1) % 2), dtype=torch.int32, device="cuda")
    need = c.ws.numel()
    buf = torch.full((need + (1 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    buf[:256].zero_()
    c.ws = buf[:need]
    c.run(c.outputs())
    assert B.moe_check_device_error(c.ws) != 0
    assert (buf[need:] == 0x5A).all()


def test_ragged_edges_do_not_read_their_neighbours():
    """K and N that end inside a tile, with NaN right behind every operand."""
    M, N, K = 70, 72, 200
    c = Lin(23, M, N, K, FP, "silu")
    out = c.outputs()
    c.run(out)

    def fenced(t):
        buf = torch.full((t.numel() + 4096,), float("nan"), dtype=t.dtype, device="cuda")
        v = buf[2048:2048 + t.numel()].view(t.shape)
        v.copy_(t)
        return buf, v

    keep = []
    for name in ("x", "w", "bias", "res", "dy"):
        buf, v = fenced(getattr(c, name))
        keep.append(buf)
        setattr(c, name, v)
    got = {}
    for n, t in c.outputs().items():
        buf, got[n] = fenced(t)
        keep.append(buf)
    c.run(got)
    for n in out:
        assert torch.equal(got[n], out[n]), n
    for buf in keep:
        assert torch.isnan(buf[:2048]).all() and torch.isnan(buf[buf.numel() - 2048:]).all()


def test_bad_offsets_are_skipped_and_reported():
    c = Lin(24, 100, 72, 64, BF, "relu", [20, 30, 40])
    good = c.outputs()
    c.run(good)
    c.off = torch.tensor([0, 20, 10, 10], dtype=torch.int32, device="cuda")       # expert 1's group runs backwards
    out = c.outputs()
    c.run(out)
    assert B.moe_check_device_error(c.ws) == B.DEVERR_BAD_OFFSETS
    assert B.moe_check_device_error(c.ws) == 0            # read and cleared
    assert torch.equal(out["y"][:20], good["y"][:20]) and (out["y"][20:] == -77).all()
    assert torch.equal(out["dw"][0], good["dw"][0]) and torch.equal(out["dx"][:20], good["dx"][:20])
    assert (out["dw"][1:] == 0).all() and (out["db"][1:] == 0).all()
    c.off = torch.tensor([0, 20, 50, 101], dtype=torch.int32, device="cuda")      # the last one ends past M
    out = c.outputs()
    c.run(out)
    assert B.moe_check_device_error(c.ws) == B.DEVERR_BAD_OFFSETS
    assert torch.equal(out["y"][:50], good["y"][:50]) and (out["y"][50:] == -77).all()
    assert (out["dw"][2] == 0).all()


def test_weights_past_32_bit_offsets():
    E, N, K = 540, 1024, 4096                             # 2.3e9 weights
    n = [0] * E
    n[0], n[511], n[512], n[539] = 3, 70, 1, 200
    M = sum(n)
    lc = B.LinearConfig(M=M, N=N, K=K, E=E, act="gelu")
    ws, off = B.alloc_linear_workspace(lc), group_offsets(n)
    w = torch.randn(E, N, K, generator=gen(1), device="cuda", dtype=BF).mul_(K ** -0.5)
    x, dy = (torch.randn(M, s, generator=gen(2), device="cuda", dtype=BF) for s in (K, N))
    y, z, dx = torch.empty(M, N, dtype=BF, device="cuda"), torch.empty(M, N, dtype=BF, device="cuda"), torch.empty_like(x)
    dw = torch.full_like(w, 9.0)
    B.moe_linear_forward(lc, x, w, y, ws, z=z, offsets=off)
    B.moe_linear_backward(lc, x, w, z, dy, ws, dx=dx, dw=dw, offsets=off)
    assert B.moe_check_device_error(ws) == 0
    lo = 0
    for e in (0, 511, 512, 539):
        rows = slice(lo, lo + n[e])
        lo += n[e]
        one = B.LinearConfig(M=n[e], N=N, K=K, act="gelu")
        out = {"y": y[rows], "z": z[rows], "dx": dx[rows], "dw": dw[e]}
        check_linear(out, x[rows], w[e], None, None, dy[rows], one, None, n[e])
    for e in range(E):
        if n[e] == 0:
            assert not dw[e].any(), e


def test_two_calls_at_once_on_two_streams():
    a, b = Lin(25, 300, 264, 520, BF, "gelu"), Lin(26, 90, 512, 1024, FP, "silu", [50, 0, 40])
    want = []
    for c in (a, b):
        out = c.outputs()
        c.run(out)
        want.append(out)
    got = [a.outputs(), b.outputs()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, out, s in zip((a, b), got, streams):
            c.run(out, stream=s)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for n in w:
            assert torch.equal(w[n], g[n]), n


@pytest.mark.parametrize("M,N,K,counts", [(128, 264, 2056, None), (40, 264, 2056, [30, 10]), (4200, 4232, 136, None),
                                          (1300, 2184, 4232, [513, 787])])
def test_large_and_split_products_replayed_from_a_graph(M, N, K, counts):
    test_replayed_from_a_graph(M, N, K, counts)


@pytest.mark.parametrize("M,N,K,counts", [(4, 512, 1024, None), (200, 264, 520, None), (600, 512, 256, [300, 0, 290]),
                                          (96, 128, 256, [4] * 24)])
def test_replayed_from_a_graph(M, N, K, counts):
    c = Lin(27, M, N, K, BF, "gelu", counts)
    want = c.outputs()
    c.run(want)
    out = c.outputs()
    c.run(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out)
    for i in range(3):
        for t in out.values():
            t.fill_(-77.0)
        c.ws[256:].fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(out[n], want[n]), (i, n)
