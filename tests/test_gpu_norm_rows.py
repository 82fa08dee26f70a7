"""Norm gradients of rows that take a block each, with several rows to a block, and of rows that
are read twice, with several to a wave: each kernel's loop over its rows, its sums for gamma and
beta over them, and their parts."""
import pytest
import torch

from block_cases import BF, F32, FP, gen, n64
from mixture_experts_layer_dispatch_amd import binding as B
from test_gpu_norm import check_backward, check_forward, inputs, nan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# a block a row (at most 512 blocks): 16-bit rows of 4104 .. 16384, fp32 rows of 2056 .. 8192; read twice
# (at most 64 parts of four waves): beyond
SHAPES = [(1100, 4104, BF, BF), (1300, 8192, BF, F32), (513, 16384, FP, FP), (1100, 2056, F32, F32), (600, 8192, F32, F32),
          (700, 16392, BF, BF), (300, 16392, FP, F32), (513, 8200, F32, F32)]


@pytest.mark.parametrize("M,H,dtype,params", SHAPES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_many_rows_to_a_block(M, H, dtype, params, kind):
    v = inputs(M + H, M, H, dtype, params)
    nc = B.NormConfig(M=M, H=H, dtype=dtype, kind=kind, params=params)
    residual = kind == "layer"
    _, h = check_forward(v, nc, residual, False)
    a = check_backward(v, nc, h, residual)
    b = check_backward(v, nc, h, residual)
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("want", [("dx",), ("dgamma",), ("dbeta",), ("dx", "dbeta"), ("dgamma", "dbeta")])
@pytest.mark.parametrize("M,H,dtype", [(600, 4104, BF), (530, 2056, F32), (300, 16392, BF), (257, 8200, F32)])
def test_each_gradient_alone(want, M, H, dtype):
    v = inputs(6, M, H, dtype, F32)
    nc = B.NormConfig(M=M, H=H, dtype=dtype, params=F32)
    check_backward(v, nc, n64(v["x"]), True, want)


@pytest.mark.parametrize("M,H", [(600, 4104), (300, 16392)])
def test_in_place(M, H):
    """dx may be dy or d_total, d_total may be dy."""
    nc = B.NormConfig(M=M, H=H)
    v = inputs(13, M, H, BF, BF)
    out, h = check_forward(v, nc, True, True)
    ws = B.alloc_norm_workspace(nc)
    for same in (False, True):
        ref = [nan(M, H, dtype=BF), nan(H, dtype=BF), nan(H, dtype=BF)]
        B.moe_norm_backward(nc, out["total"], v["gamma"], out["rstd"], v["dy"], ref[0], ws, mean=out["mean"],
                            d_total=v["dy"] if same else v["dt"], dgamma=ref[1], dbeta=ref[2])
        for name in ("dy", "dt"):
            if same and name == "dt":
                continue
            w = {n: t.clone() for n, t in v.items()}
            dg, db = nan(H, dtype=BF), nan(H, dtype=BF)
            B.moe_norm_backward(nc, out["total"], v["gamma"], out["rstd"], w["dy"], w[name], ws, mean=out["mean"],
                                d_total=w["dy"] if same else w["dt"], dgamma=dg, dbeta=db)
            assert torch.equal(w[name], ref[0]) and torch.equal(dg, ref[1]) and torch.equal(db, ref[2])


@pytest.mark.parametrize("M,H", [(1030, 4104), (520, 16392)])
def test_graph(M, H):
    nc = B.NormConfig(M=M, H=H, kind="rms")
    v = inputs(14, M, H, BF, BF)
    ws, y, rstd, dx, dg = B.alloc_norm_workspace(nc), nan(M, H, dtype=BF), nan(M), nan(M, H, dtype=BF), nan(H, dtype=BF)

    def step():
        B.moe_norm_forward(nc, v["x"], v["gamma"], y, rstd=rstd)
        B.moe_norm_backward(nc, v["x"], v["gamma"], rstd, v["dy"], dx, ws, dgamma=dg)

    step()
    first = [t.clone() for t in (y, rstd, dx, dg)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (y, rstd, dx, dg):
            t.fill_(-3)
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, rstd, dx, dg), first))
