"""GPU parity of permute / unpermute and their gradients against the 64-bit
reference: one token, one expert, all experts, odd counts, several macrobatches,
rows that need 64-bit offsets, bad rows, other streams, captured graphs."""
import numpy as np
import pytest
import torch

from block_cases import BF, F32, FP, STEP, TINY, U, assert_within, gen, n64, randn, schedule, sum_err
from mixture_experts_layer_dispatch_amd import binding as B
from oracle import blocks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# T, E, k, H, macrobatch
SHAPES = [(1, 1, 1, 128, 0), (1, 512, 10, 4096, 0), (5, 3, 3, 128, 0), (100, 7, 3, 256, 0), (64, 32, 32, 128, 0),
          (333, 40, 9, 640, 0), (256, 16, 4, 1152, 64), (37, 1024, 17, 384, 0)]


class Rows:
    def __init__(self, seed, T, E, k, H, macrobatch, dtype):
        self.cfg, self.sched, self.ws = schedule(seed, T, E, k, H, macrobatch)
        g = gen(seed + 1)
        self.x, self.res, self.dy = (randn(g, (T, H), dtype) for _ in range(3))
        self.o = randn(g, (T * k, H), dtype)
        self.dtype = dtype

    def outputs(self):
        c, dt = self.cfg, self.dtype
        nan = float("nan")
        return {"xs": torch.full((c.S, c.H), nan, dtype=dt, device="cuda"),
                "dx": torch.full((c.T, c.H), nan, dtype=dt, device="cuda"),
                "y": torch.full((c.T, c.H), nan, dtype=dt, device="cuda"),
                "y_res": torch.full((c.T, c.H), nan, dtype=dt, device="cuda"),
                "do": torch.full((c.S, c.H), nan, dtype=dt, device="cuda"),
                "dw": torch.full((c.T, c.k), nan, device="cuda"),
                "dl": torch.full((c.T, c.E), nan, device="cuda")}

    def run(self, out, stream=None):
        a = (self.cfg, self.sched)
        B.moe_permute_forward(*a, self.x, out["xs"], self.ws, stream=stream)
        B.moe_permute_backward(*a, self.o, out["dx"], self.ws, stream=stream)
        B.moe_unpermute_forward(*a, self.o, out["y"], self.ws, stream=stream)
        B.moe_unpermute_forward(*a, self.o, out["y_res"], self.ws, residual=self.res, stream=stream)
        B.moe_unpermute_backward(*a, self.o, self.dy, out["do"], out["dw"], self.ws, d_logits=out["dl"],
                                 stream=stream)

    def check(self, out):
        c, u, tiny = self.cfg, U[self.dtype], TINY[self.dtype]
        row, w, idx = (self.sched[n].cpu().numpy() for n in ("row_of_slot", "topk_w", "topk_idx"))
        o, dy, res = n64(self.o), n64(self.dy), n64(self.res)
        np.testing.assert_array_equal(n64(out["xs"]), blocks.permute(n64(self.x), row, c.k))
        ones = np.ones((c.T, c.k))

        def near(name, ref, mag):
            assert_within(name, out[name], ref, u * np.abs(ref) + sum_err(c.k + 1, mag) + tiny)

        near("dx", blocks.permute_backward(o, row, c.k), blocks.unpermute(np.abs(o), row, ones))
        near("y", blocks.unpermute(o, row, w), blocks.unpermute(np.abs(o), row, w))
        near("y_res", blocks.unpermute(o, row, w, res), blocks.unpermute(np.abs(o), row, w, np.abs(res)))
        do, dw, dl = blocks.unpermute_backward(o, dy, row, w, idx, c.E)
        assert_within("do", out["do"], do, (u + STEP) * np.abs(do) + tiny)
        mag = blocks.unpermute_backward(np.abs(o), np.abs(dy), row, w, idx, c.E)[1]
        assert_within("dw", out["dw"], dw, sum_err(c.H, mag))
        # d_logit = w (dw - sum w dw): dw's error and the sum's, both scaled by w
        err = sum_err(c.H, mag) + sum_err(c.k + 4, np.abs(dw) + (w * np.abs(dw)).sum(1, keepdims=True))
        tol = np.zeros((c.T, c.E))
        np.put_along_axis(tol, idx.astype(np.int64), w * (err + (w * err).sum(1, keepdims=True)) + 1e-37, axis=1)
        assert_within("dl", out["dl"], dl, tol)
        assert B.moe_check_device_error(self.ws) == 0


@pytest.mark.parametrize("dtype", [BF, FP, F32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,E,k,H,macro", SHAPES)
def test_rows_to_experts_and_back(T, E, k, H, macro, dtype):
    r = Rows(11, T, E, k, H, macro, dtype)
    out = r.outputs()
    r.run(out)
    r.check(out)
    again = r.outputs()
    r.run(again)
    for n in out:
        assert torch.equal(out[n], again[n]), n           # the order of every sum is fixed


def test_residual_may_be_the_output():
    r = Rows(12, 100, 7, 3, 256, 0, BF)
    want = torch.empty_like(r.res)
    B.moe_unpermute_forward(r.cfg, r.sched, r.o, want, r.ws, residual=r.res)
    y = r.res.clone()
    B.moe_unpermute_forward(r.cfg, r.sched, r.o, y, r.ws, residual=y)
    assert torch.equal(y, want)


def test_without_logit_gradients_and_with_a_bare_error_word():
    r = Rows(13, 50, 9, 4, 128, 0, BF)
    out, ws = r.outputs(), B.alloc_error_word()
    sched = {n: r.sched[n] for n in ("row_of_slot", "topk_w")}
    B.moe_unpermute_backward(r.cfg, sched, r.o, r.dy, out["do"], out["dw"], ws)
    full = r.outputs()
    r.run(full)
    assert torch.equal(out["do"], full["do"]) and torch.equal(out["dw"], full["dw"])
    assert B.moe_check_device_error(ws) == 0


def test_infinities_and_nan_stay_in_their_rows_and_columns():
    r = Rows(14, 20, 5, 2, 128, 0, BF)
    row = r.sched["row_of_slot"].view(20, 2).long()
    clean = r.outputs()
    r.run(clean)
    r.o[row[3, 0], 7] = float("inf")
    r.o[row[4, 1], 9] = float("nan")
    out = r.outputs()
    r.run(out)
    y, ref = out["y"], clean["y"].clone()
    assert y[3, 7] == float("inf") and torch.isnan(y[4, 9])
    ref[3, 7], ref[4, 9] = y[3, 7], y[4, 9]
    assert torch.equal(y.nan_to_num(5.0), ref.nan_to_num(5.0))
    keep = [t for t in range(20) if t not in (3, 4)]
    assert torch.equal(out["dw"][keep], clean["dw"][keep])
    assert torch.equal(out["dl"][keep], clean["dl"][keep])


def test_rows_outside_the_table_are_skipped_and_reported():
    r = Rows(15, 40, 6, 3, 128, 0, F32)
    clean = r.outputs()
    r.run(clean)
    good = r.sched["row_of_slot"].clone()
    bad = good.clone()
    bad[5], bad[70] = 120, -3                             # S = 120
    r.sched["row_of_slot"] = bad
    out = r.outputs()
    r.run(out)
    assert B.moe_check_device_error(r.ws) == B.DEVERR_BAD_ROW
    assert B.moe_check_device_error(r.ws) == 0            # read and cleared
    for s in (5, 70):
        assert torch.isnan(out["xs"][good[s].long()]).all()       # left as it was
        assert torch.isnan(out["do"][good[s].long()]).all()
        assert out["dw"].view(-1)[s] == 0
    rows = [int(v) for i, v in enumerate(good.tolist()) if i not in (5, 70)]
    assert torch.equal(out["xs"][rows], clean["xs"][rows])
    tokens = [t for t in range(40) if t not in (5 // 3, 70 // 3)]
    assert torch.equal(out["y"][tokens], clean["y"][tokens])


def test_rows_past_32_bit_offsets():
    """S * H = 2.3e9 elements, on the framework's own schedule."""
    T, E, k, H = 70000, 64, 8, 4096
    cfg = B.Config(T=T, H=H, I=128, E=E, k=k)
    sched = B.alloc_schedule(cfg)
    B.moe_schedule_noalloc(cfg, torch.randn(T, E, generator=gen(3), device="cuda"), sched)
    ws = B.alloc_error_word()
    x = torch.randn(T, H, generator=gen(4), device="cuda", dtype=BF)
    xs = torch.zeros(T * k, H, dtype=BF, device="cuda")
    B.moe_permute_forward(cfg, sched, x, xs, ws)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    B.moe_unpermute_forward(cfg, sched, xs, y, ws)
    B.moe_permute_backward(cfg, sched, xs, dx, ws)
    do, dw = torch.zeros_like(xs), torch.empty(T, k, device="cuda")
    B.moe_unpermute_backward(cfg, sched, xs, x, do, dw, ws)
    for rows in torch.arange(T * k, device="cuda").split(T):
        t = sched["slot_of_row"][rows].long() // k
        assert torch.equal(xs[rows], x[t])
        w = sched["topk_w"].view(-1)[sched["slot_of_row"][rows].long()]
        assert torch.equal(do[rows], (w[:, None] * x[t].float()).to(BF))
    # every expert row is the token's own: the weights sum to one, the gradient to k copies
    xf = x.float()
    assert ((y.float() - xf).abs() <= (U[BF] + 16 * STEP) * xf.abs()).all()
    assert ((dx.float() - k * xf).abs() <= (U[BF] + 16 * STEP) * k * xf.abs()).all()
    n = (xf * xf).sum(1, keepdim=True)
    assert ((dw - n).abs() <= (2 * H + 4) * STEP * n).all()
    assert B.moe_check_device_error(ws) == 0


def test_on_another_stream_and_replayed_from_a_graph():
    r = Rows(16, 200, 24, 5, 384, 0, BF)
    want = r.outputs()
    r.run(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = r.outputs()
    torch.cuda.synchronize()
    r.run(out, stream=side)
    side.synchronize()
    for n in want:
        assert torch.equal(out[n], want[n]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.run(out)
    for _ in range(3):
        for t in out.values():
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(out[n], want[n]), n


def test_more_tokens_than_one_grid_dimension_takes():
    """k = 1, 2^24 + 5 tokens of 640: more than 2^32 threads in every launch."""
    T, H, step = (1 << 24) + 5, 640, 1 << 21
    cfg, ws = B.Config(T=T, H=H, I=128, E=4, k=1), B.alloc_error_word()
    row = (T - 1 - torch.arange(T, device="cuda")).to(torch.int32)          # row(t) = T - 1 - t
    sched = {"row_of_slot": row, "topk_w": (torch.arange(T, device="cuda") % 7 - 3).float().view(T, 1)}
    marks = (torch.arange(T, device="cuda") % 251).to(BF).view(T, 1)        # exact in bf16, also times -3 .. 3
    col = torch.arange(H, device="cuda") % 2 == 0
    a, b = torch.empty(T, H, dtype=BF, device="cuda"), torch.empty(T, H, dtype=BF, device="cuda")
    for i in range(0, T, step):
        a[i:i + step] = torch.where(col, marks[i:i + step], 1)

    def check(out, want):
        for i in range(0, T, step):
            assert torch.equal(out[i:i + step], want(torch.arange(i, min(i + step, T), device="cuda"))), i

    def rows(t):
        return torch.where(col, marks[t], 1).to(BF)

    def weighted(t):
        return (rows(t).float() * sched["topk_w"][t]).to(BF)

    B.moe_permute_forward(cfg, sched, a, b, ws)
    check(b, lambda r: rows(T - 1 - r))
    a.fill_(-77)
    B.moe_permute_backward(cfg, sched, b, a, ws)
    check(a, rows)
    a.fill_(-77)
    B.moe_unpermute_forward(cfg, sched, b, a, ws)
    check(a, weighted)
    for i in range(0, T, step):
        a[i:i + step] = 1                                                    # dy: the weights' gradient counts the row
    c, dw = torch.empty_like(a), torch.empty(T, 1, device="cuda")
    B.moe_unpermute_backward(cfg, sched, b, a, c, dw, ws)
    check(c, lambda r: sched["topk_w"][T - 1 - r].to(BF).expand(-1, H))
    assert torch.equal(dw, marks.float() * 320 + 320)
    assert B.moe_check_device_error(ws) == 0
