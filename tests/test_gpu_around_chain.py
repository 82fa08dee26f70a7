"""Norm, router, routing with groups, schedule, experts and combine together, as a
block of a model uses them: answering with 4-bit experts, and a training step
with its backward pass.  Each step is checked against the 64-bit reference on the
inputs it had, whole steps against a second run and replayed graphs bit for bit."""
import numpy as np
import pytest
import torch

from block_cases import ACT_ERR, ACT_SLOPE, BF, F32, STEP, TINY, U, assert_within, gen, n64, randn, sum_err
from mixture_experts_layer_dispatch_amd import binding as B
from oracle import around, blocks

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -24
u, tiny = U[BF], TINY[BF]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def new(*s, dtype=BF):
    return torch.full(s, float("nan"), dtype=dtype, device="cuda")


class Block:
    """A pre-norm block with experts of two projections, trained in bf16 (w1, w2) or served in 4 bits."""

    def __init__(self, T, H, F, E, k, seed, kind="rms", score="sigmoid", macrobatch=0):
        g = gen(seed)
        self.cfg = B.Config(T=T, H=H, I=128, E=E, k=k, macrobatch=macrobatch)
        self.route = B.RouteConfig(score=score, n_group=4, topk_group=2, group_top=2, scale=1.5)
        self.nc = B.NormConfig(M=T, H=H, kind=kind)
        S, Sm = T * k, self.cfg.M * k
        self.up = B.LinearConfig(M=Sm, N=F, K=H, E=E, act="silu")
        self.down = B.LinearConfig(M=Sm, N=H, K=F, E=E)
        self.up4 = B.LinearW4Config(M=Sm, N=F, K=H, E=E, group=64, act="silu")
        self.down4 = B.LinearW4Config(M=Sm, N=H, K=F, E=E, group=32)
        self.x, self.skip, self.dy, self.dskip = (randn(g, (T, H), BF) for _ in range(4))
        self.gamma = (1 + randn(g, (H,), F32, 0.2)).to(BF)
        self.beta = randn(g, (H,), BF, 0.2) if kind == "layer" else None
        self.wr, self.balance = randn(g, (E, H), BF, H ** -0.5), randn(g, (E,), F32, 0.02)
        self.w1, self.w2 = randn(g, (E, F, H), BF, H ** -0.5), randn(g, (E, H, F), BF, F ** -0.5)
        self.q1, self.q2 = B.alloc_linear_w4_weights(self.up4, zeros=True), B.alloc_linear_w4_weights(self.down4)
        B.moe_linear_w4_quantize(self.up4, self.w1, **self.q1)
        B.moe_linear_w4_quantize(self.down4, self.w2, **self.q2)
        self.ws, self.wn = B.alloc_workspace(self.cfg), B.alloc_norm_workspace(self.nc)
        self.wu, self.wd = B.alloc_linear_workspace(self.up), B.alloc_linear_workspace(self.down)
        self.wu4, self.wd4 = B.alloc_linear_w4_workspace(self.up4), B.alloc_linear_w4_workspace(self.down4)
        self.sched = B.alloc_schedule(self.cfg)
        self.t = {"total": new(T, H), "n": new(T, H), "rstd": new(T, dtype=F32), "logits": new(T, E, dtype=F32),
                  "xs": new(S, H), "h": new(S, F), "o": new(S, H), "y": new(T, H), "scores": new(T, E, dtype=F32)}
        if kind == "layer":
            self.t["mean"] = new(T, dtype=F32)

    def begin(self):
        t = self.t
        B.moe_norm_forward(self.nc, self.x, self.gamma, t["n"], beta=self.beta, residual=self.skip, total=t["total"],
                           mean=t.get("mean"), rstd=t["rstd"])
        B.moe_router_forward(self.cfg, t["n"], self.wr, t["logits"])
        B.moe_route_forward(self.cfg, self.route, t["logits"], self.sched, bias=self.balance, scores=t["scores"])
        B.moe_schedule_from_topk(self.cfg, self.sched, self.ws)
        B.moe_permute_forward(self.cfg, self.sched, t["n"], t["xs"], self.ws)

    def serve(self):
        self.begin()
        t, Sm = self.t, self.cfg.M * self.cfg.k
        for m in range(self.cfg.n_macro):
            r, off = slice(m * Sm, (m + 1) * Sm), self.sched["offsets"][m]
            B.moe_linear_w4_forward(self.up4, t["xs"][r], y=t["h"][r], ws=self.wu4, offsets=off, **self.q1)
            B.moe_linear_w4_forward(self.down4, t["h"][r], y=t["o"][r], ws=self.wd4, offsets=off, **self.q2)
        B.moe_unpermute_forward(self.cfg, self.sched, t["o"], t["y"], self.ws, residual=t["total"])

    def train(self):
        if "z" not in self.t:
            T, H, E, k = self.cfg.T, self.cfg.H, self.cfg.E, self.cfg.k
            S, F = T * k, self.up.N
            self.t.update(z=new(S, F), do=new(S, H), dtok=new(T, k, dtype=F32), dh=new(S, F), dw2=new(E, H, F),
                          dxs=new(S, H), dw1=new(E, F, H), dn=new(T, H), dl=new(T, E, dtype=F32), dwr=new(E, H),
                          dx=new(T, H), dgamma=new(H))
            if self.nc.kind == "layer":
                self.t["dbeta"] = new(H)
            self.dscores = (0.01 * self.balance / T).expand(T, E).contiguous()
        self.begin()
        t, c, s, off = self.t, self.cfg, self.sched, self.sched["offsets"][0]
        B.moe_linear_forward(self.up, t["xs"], self.w1, t["h"], self.wu, z=t["z"], offsets=off)
        B.moe_linear_forward(self.down, t["h"], self.w2, t["o"], self.wd, offsets=off)
        B.moe_unpermute_forward(c, s, t["o"], t["y"], self.ws, residual=t["total"])
        B.moe_unpermute_backward(c, s, t["o"], self.dy, t["do"], t["dtok"], self.ws)
        B.moe_linear_backward(self.down, t["h"], self.w2, None, t["do"], self.wd, dx=t["dh"], dw=t["dw2"], offsets=off)
        B.moe_linear_backward(self.up, t["xs"], self.w1, t["z"], t["dh"], self.wu, dx=t["dxs"], dw=t["dw1"], offsets=off)
        B.moe_permute_backward(c, s, t["dxs"], t["dn"], self.ws)
        B.moe_route_backward(c, self.route, t["logits"], s, t["dtok"], t["dl"], self.ws, d_scores=self.dscores)
        B.moe_router_backward(c, t["n"], self.wr, t["dl"], t["dn"], t["dwr"], self.ws)
        # the skip connection's gradient is the output's, beside that of a later block
        B.moe_norm_backward(self.nc, t["total"], self.gamma, t["rstd"], t["dn"], t["dx"], self.wn, mean=t.get("mean"),
                            d_total=self.dy, dgamma=t["dgamma"], dbeta=t.get("dbeta"))


def check_begin(m):
    t, layer = m.t, m.nc.kind == "layer"
    h = n64(m.x) + n64(m.skip)
    assert_within("total", t["total"], h, (u + HALF) * (1 + u) * np.abs(h) + tiny)
    h, H = n64(t["total"]), m.cfg.H
    y, mean, rstd = around.norm(h, n64(m.gamma), n64(m.beta) if layer else None, m.nc.kind)
    d = (H / 64 + 40) * STEP
    dm = d * np.abs(h).mean(1, keepdims=True)
    xh = np.abs(h - mean[:, None]) * rstd[:, None]
    tol = np.abs(n64(m.gamma)) * (rstd[:, None] * dm + xh * d) + d * np.abs(y)
    assert_within("n", t["n"], y, (tol + u * np.abs(y)) * (1 + u) + tiny)
    n, wr = n64(t["n"]), n64(m.wr)
    assert_within("logits", t["logits"], n @ wr.T, sum_err(H, np.abs(n) @ np.abs(wr).T))
    r = m.route
    idx, w, s = around.route(n64(t["logits"]), m.cfg.k, r.score, n64(m.balance), r.n_group, r.topk_group, r.group_top,
                             r.renorm, r.scale)
    np.testing.assert_array_equal(m.sched["topk_idx"].cpu().numpy(), idx)
    assert_within("w", m.sched["topk_w"], w, 64 * HALF * w)
    assert_within("scores", t["scores"], s, 64 * HALF * s)
    row = m.sched["row_of_slot"].cpu().numpy()
    np.testing.assert_array_equal(np.sort(row), np.arange(len(row)))
    np.testing.assert_array_equal(n64(t["xs"]), blocks.permute(n, row, m.cfg.k))
    return row


def linear_tol(ref, lin, mag, K, act):
    tol = ACT_SLOPE * sum_err(K + 4, mag) + (ACT_ERR * np.maximum(np.abs(lin), 1) if act else 0)
    return (tol + u * np.abs(ref)) * (1 + 2 * u) + tiny


def replayed(m, step, names):
    step()
    first = {n: m.t[n].clone() for n in names}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for n in names:
            m.t[n].fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(m.t[n], first[n]), n


@pytest.mark.parametrize("T,H,F,E,k,macrobatch", [(1, 256, 64, 8, 2, 0), (5, 128, 192, 32, 6, 0),
                                                  (300, 256, 160, 16, 3, 0), (64, 128, 96, 12, 4, 16)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_serving_with_4_bit_experts(T, H, F, E, k, macrobatch, kind):
    m = Block(T, H, F, E, k, 41, kind, macrobatch=macrobatch)
    m.serve()
    for ws in (m.ws, m.wu4, m.wd4):
        assert B.moe_check_device_error(ws) == 0
    row, t = check_begin(m), m.t
    Sm = m.cfg.M * k
    off = np.concatenate([n64(o)[:-1] + i * Sm for i, o in enumerate(m.sched["offsets"])] + [[T * k]]).astype(int)
    for name, src, q, K, act in (("h", "xs", m.q1, H, "silu"), ("o", "h", m.q2, F, "none")):
        v = {n: c.cpu().numpy() if c.dtype == torch.uint8 else n64(c) for n, c in q.items()}
        v = {n: np.concatenate([c] * m.cfg.n_macro) for n, c in v.items()}        # a group per macrobatch and expert
        ref, lin, mag = around.linear_w4(n64(t[src]), v["codes"], v["scales"], v.get("zeros"), None, None, act, off)
        assert_within(name, t[name], ref, linear_tol(ref, lin, mag, K + K // 32, act == "silu"))
    o, w, total = n64(t["o"]), n64(m.sched["topk_w"]), n64(t["total"])
    y = blocks.unpermute(o, row, w, total)
    mag = blocks.unpermute(np.abs(o), row, np.abs(w), np.abs(total))
    assert_within("y", t["y"], y, (sum_err(k + 1, mag) + u * np.abs(y)) * (1 + 2 * u) + tiny)
    replayed(m, m.serve, list(t))


@pytest.mark.parametrize("T,H,F,E,k,score", [(200, 128, 96, 12, 3, "sigmoid"), (3, 256, 64, 40, 5, "softmax"),
                                             (130, 128, 160, 8, 4, "softmax")])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_training_step(T, H, F, E, k, score, kind):
    m = Block(T, H, F, E, k, 43, kind, score)
    m.train()
    for ws in (m.ws, m.wu, m.wd):
        assert B.moe_check_device_error(ws) == 0
    row, v = check_begin(m), {n: n64(t) for n, t in m.t.items()}
    w1, w2, dy = n64(m.w1), n64(m.w2), n64(m.dy)
    off, w = m.sched["offsets"][0].tolist(), n64(m.sched["topk_w"])
    idx = m.sched["topk_idx"].cpu().numpy()
    h, z, mag = blocks.linear(v["xs"], w1, None, None, "silu", off)
    assert_within("h", m.t["h"], h, linear_tol(h, z, mag, H, True))
    o, _, mag = blocks.linear(v["h"], w2, None, None, "none", off)
    assert_within("o", m.t["o"], o, linear_tol(o, o, mag, F, False))
    do, dtok, _ = blocks.unpermute_backward(v["o"], dy, row, w, idx, E)
    dmag = blocks.unpermute_backward(np.abs(v["o"]), np.abs(dy), row, w, idx, E)[1]
    assert_within("dtok", m.t["dtok"], dtok, sum_err(H, dmag))
    # the router's gradient: the weights' and the balance term's
    r = m.route
    dl = around.route_backward(v["logits"], idx, v["dtok"], score, r.renorm, r.scale, n64(m.dscores))
    share = around.chosen_share(v["logits"], idx, score)
    size = r.scale * share * (np.abs(v["dtok"]) + (share * np.abs(v["dtok"])).sum(1, keepdims=True))
    full = around.scores(v["logits"], score) * np.abs(n64(m.dscores))
    np.add.at(full, (np.arange(T)[:, None], idx), size)
    full = full + (around.scores(v["logits"], score) * full.sum(1, keepdims=True) if score == "softmax" else 0)
    assert_within("dl", m.t["dl"], dl, 2 * (E / 64 + 22 + k) * HALF * full + 2.0 ** -126)
    # back through the norm, where the skip connection's gradient joins
    layer = kind == "layer"
    dx, dgamma, dbeta = around.norm_backward(v["total"], n64(m.gamma), v.get("mean"), v["rstd"], v["dn"], kind, dy)
    xh = np.abs(v["total"] - (v["mean"][:, None] if layer else 0)) * v["rstd"][:, None]
    g = np.abs(v["dn"] * n64(m.gamma))
    d = (H / 64 + 40) * STEP
    tol = v["rstd"][:, None] * d * (g + g.mean(1, keepdims=True) + xh * (1 + (g * xh).mean(1, keepdims=True))) + d * np.abs(dy)
    assert_within("dx", m.t["dx"], dx, (tol + u * np.abs(dx)) * (1 + u) + tiny)
    assert_within("dgamma", m.t["dgamma"], dgamma,
                  (sum_err(T, (np.abs(v["dn"]) * xh).sum(0)) + u * np.abs(dgamma)) * (1 + u) + tiny)
    if layer:
        assert_within("dbeta", m.t["dbeta"], dbeta,
                      (sum_err(T, np.abs(v["dn"]).sum(0)) + u * np.abs(dbeta)) * (1 + u) + tiny)
    replayed(m, m.train, list(m.t))


def test_the_layer_itself_takes_the_routing():
    """moe_forward and moe_backward on a table from moe_route_forward and moe_schedule_from_topk: with the
    layer's own kind of routing the same bits, its router gradient from dw."""
    T, H, I, E, k = 48, 256, 128, 16, 3
    cfg, g = B.Config(T=T, H=H, I=I, E=E, k=k), gen(44)
    logits, x, dy = torch.randn(T, E, generator=g, device="cuda"), randn(g, (T, H), BF), randn(g, (T, H), BF)
    w = {"w_gate": randn(g, (E, I, H), BF, H ** -0.5), "w_up": randn(g, (E, I, H), BF, H ** -0.5),
         "w_down": randn(g, (E, H, I), BF, I ** -0.5)}
    out = []
    for own in (False, True):
        ws, sched, saved, grads = B.alloc_workspace(cfg), B.alloc_schedule(cfg), B.alloc_saved(cfg), B.alloc_grads(cfg)
        y, dx, dw, dl = new(T, H), new(T, H), new(T, k, dtype=F32), new(T, E, dtype=F32)
        if own:
            B.moe_schedule(cfg, logits, sched, ws)
        else:
            B.moe_route_forward(cfg, B.RouteConfig(), logits, sched)
            B.moe_schedule_from_topk(cfg, sched, ws)
        wts = sched["topk_w"]
        if own:
            wts.copy_(out[0][0])                              # (half a step apart: take the same)
        B.moe_forward(cfg, sched, x, w, y, saved, ws)
        B.moe_backward(cfg, sched, saved, x, w, dy, dx, grads, dw, dl if own else None, ws)
        if not own:
            B.moe_route_backward(cfg, B.RouteConfig(), logits, sched, dw, dl, ws)
        assert B.moe_check_device_error(ws) == 0
        out.append([wts.clone(), y, dx, dw, *grads.values(), dl])
    for a, b in zip(out[0][:-1], out[1][:-1]):
        assert torch.equal(a, b)
    mag = (out[0][0] * out[0][3].abs()).sum(1, keepdim=True) * 2
    assert ((out[0][-1] - out[1][-1]).abs() <= 40 * HALF * mag).all()
