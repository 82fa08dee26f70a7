"""Cases, plain forms and calls of the layer's building-block operators:

  permute     token rows copied to their experts' rows, and the gradient
  unpermute   expert rows summed back to tokens with the router weights and a
              residual, and the gradients (rows, weights, router logits)
  linear      y = act(x W^T + b) + residual, dense or grouped by expert, and
              the gradients of x, W and b

``listed()`` are fixed cases, ``draw(rng)`` gives more of the same ranges,
``prepare`` makes a case's inputs from a seed, ``run`` computes one pass: in
elementary torch operations (``own`` false), or through the package's entry
points (``own`` true).  ``exact`` computes the same from the definition in 64
bits, ``work`` says what a pass has to move and compute.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # four tokens of a decode step go to ten of 512 experts: latency
        dict(name="permute_fwd_decode", op="permute_fwd", T=4, H=4096, E=512, k=10, dtype="bf16"),
        # one macrobatch of a long training stream, dispatched
        dict(name="permute_fwd_t16384", op="permute_fwd", T=16384, H=4096, E=512, k=10, dtype="bf16"),
        # the input gradient of a 2048-token training step, back at its tokens
        dict(name="permute_bwd_t2048", op="permute_bwd", T=2048, H=4096, E=512, k=10, dtype="bf16"),
        # the combine of a 2048-token step with the skip connection added
        dict(name="unpermute_fwd_t2048", op="unpermute_fwd", T=2048, H=4096, E=512, k=10, dtype="bf16",
             residual=True),
        # the combine's backward for one macrobatch, down to the router logits
        dict(name="unpermute_bwd_t16384", op="unpermute_bwd", T=16384, H=4096, E=512, k=10, dtype="bf16"),
        # a small layer's combine backward in fp32, odd token and expert counts
        dict(name="unpermute_bwd_odd_fp32", op="unpermute_bwd", T=333, H=384, E=7, k=3, dtype="fp32"),
        # a projection of four decoded tokens: the weight is read once, latency counts
        dict(name="linear_fwd_decode", op="linear_fwd", M=4, N=4096, K=4096, E=0, dtype="bf16", act="silu",
             bias=True, residual=True, keep=False),
        # a dense projection of one macrobatch in training (pre-activation kept)
        dict(name="linear_fwd_m16384", op="linear_fwd", M=16384, N=4096, K=4096, E=0, dtype="bf16", act="gelu",
             bias=True, residual=False, keep=True),
        # 16 decoded tokens' 160 rows at 512 experts: the experts hit are streamed
        dict(name="linear_fwd_e512_decode", op="linear_fwd", M=160, N=1024, K=4096, E=512, dtype="bf16",
             act="gelu_tanh", bias=True, residual=False, keep=False),
        # the 2048-token layer's first projection, about 40 rows an expert
        dict(name="linear_fwd_e512_t2048", op="linear_fwd", M=20480, N=1024, K=4096, E=512, dtype="bf16", act="gelu",
             bias=True, residual=False, keep=True),
        # an expert-parallel share's backward: 8 experts of about 2560 rows
        dict(name="linear_bwd_e8", op="linear_bwd", M=20480, N=1024, K=4096, E=8, dtype="bf16", act="relu", bias=True),
        # a dense layer's backward at sizes that fill no tile, fp16
        dict(name="linear_bwd_odd_fp16", op="linear_bwd", M=1111, N=1000, K=1544, E=0, dtype="fp16", act="silu",
             bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["permute_fwd", "permute_bwd", "unpermute_fwd", "unpermute_bwd", "linear_fwd", "linear_bwd"])
    if op.startswith("linear"):
        grouped = rng.random() < 0.5
        # rows and columns of 16 bytes: multiples of 8 elements, tile multiples and not
        N, K = (8 * _log(rng, 8, 1024 if not grouped else 256) for _ in range(2))
        E = _log(rng, 1, 512) if grouped else 0
        M = _log(rng, 1, 16384)
        while M * N * K > 16384 * 4096 * 4096:
            M = (M + 1) // 2
        c = dict(op=op, M=M, N=N, K=K, E=E, dtype=rng.choice(["bf16", "bf16", "fp16"]),
                 act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), bias=rng.random() < 0.7)
        if grouped:
            c["zipf"] = E <= 64 and rng.random() < 0.5
        if op == "linear_fwd":
            c.update(residual=rng.random() < 0.5, keep=rng.random() < 0.5)
        return c
    E = _log(rng, 1, 1024)
    k = rng.randint(1, min(E, 16))
    H = 128 * _log(rng, 1, 64)
    T = _log(rng, 1, 16384)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    while T * k * H * SIZE[dtype] > 16384 * 10 * 4096 * 2:
        T = (T + 1) // 2
    c = dict(op=op, T=T, H=H, E=E, k=k, dtype=dtype)
    if op == "unpermute_fwd":
        c["residual"] = rng.random() < 0.5
    return c


def work(case):
    s = SIZE[case["dtype"]]
    if case["op"].startswith("linear"):
        M, N, K, E = case["M"], case["N"], case["K"], case["E"]
        # grouped: the weights of experts without rows are not read (but their gradients are written)
        hit = min(E, M) if E else 1
        if E > 0 and not case.get("zipf"):
            hit = E * (1.0 - (1.0 - 1.0 / E) ** M)
        w, b = hit * N * K * s, hit * N * s if case["bias"] else 0
        if case["op"] == "linear_fwd":
            b += w + M * K * s + M * N * s * (1 + bool(case["residual"]) + bool(case["keep"]))
            return {"bytes": b, "flops": 2.0 * M * N * K}
        # x, dy and z in; dx, dW and db out
        dz = M * N * s * (1 if case["act"] == "none" else 2)
        out = max(E, 1) * (N * K * s + (N * s if case["bias"] else 0))
        return {"bytes": w + 2 * M * K * s + dz + out, "flops": 4.0 * M * N * K}
    T, H, E, k = case["T"], case["H"], case["E"], case["k"]
    S = T * k
    if case["op"] in ("permute_fwd", "permute_bwd"):
        return {"bytes": (T + S) * H * s + 4 * S, "flops": S * H}
    if case["op"] == "unpermute_fwd":
        return {"bytes": (T * (2 if case["residual"] else 1) + S) * H * s + 8 * S, "flops": 2.0 * S * H}
    return {"bytes": (T + 2 * S) * H * s + 16 * S + 4 * T * E, "flops": 3.0 * S * H}


# ------------------------------------------------------------------ inputs
def _randn(g, shape, dtype, std=1.0):
    t = torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[dtype])
    return t if std == 1.0 else t.mul_(std)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s, dt = dict(case), case["dtype"]
    if case["op"].startswith("linear"):
        M, N, K, E = case["M"], case["N"], case["K"], case["E"]
        lead = (E,) if E else ()
        s["x"] = _randn(g, (M, K), dt)
        s["w"] = _randn(g, (*lead, N, K), dt, K ** -0.5)
        s["bias_t"] = _randn(g, (*lead, N), dt, 0.5) if case["bias"] else None
        s["offsets"], s["most"] = None, M
        if E:
            p = torch.ones(E, device="cuda")
            if case.get("zipf"):
                p = torch.arange(1, E + 1, device="cuda").float() ** -1.1
            of = torch.multinomial(p, M, replacement=True, generator=g)
            n = torch.bincount(of, minlength=E)
            s["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
            s["most"] = int(n.max())
        if case["op"] == "linear_fwd":
            s["res"] = _randn(g, (M, N), dt) if case["residual"] else None
        else:
            s["z"] = _randn(g, (M, N), dt)
            s["dy"] = _randn(g, (M, N), dt)
        return s
    T, H, E, k = case["T"], case["H"], case["E"], case["k"]
    S = T * k
    # the schedule of random router logits: a token's k best experts, rows
    # grouped by expert, a group's rows in slot order
    v, idx = torch.randn((T, E), generator=g, device="cuda").topk(k, dim=1)
    of = idx.reshape(-1)
    slot_of_row = torch.sort(of, stable=True).indices
    row_of_slot = torch.empty_like(slot_of_row)
    row_of_slot[slot_of_row] = torch.arange(S, device="cuda")
    n = torch.bincount(of, minlength=E)
    i32 = torch.int32
    s["sched"] = {"topk_idx": idx.to(i32), "topk_w": torch.softmax(v, 1), "counts": n.view(1, E).to(i32),
                  "offsets": torch.cat([n.new_zeros(1), n.cumsum(0)]).view(1, E + 1).to(i32),
                  "mini_counts": n.view(1, E, 1).to(i32), "row_of_slot": row_of_slot.to(i32),
                  "slot_of_row": slot_of_row.to(i32)}
    if case["op"] == "permute_fwd":
        s["x"] = _randn(g, (T, H), dt)
    elif case["op"] == "permute_bwd":
        s["dxs"] = _randn(g, (S, H), dt)
    else:
        s["o"] = _randn(g, (S, H), dt)
        if case["op"] == "unpermute_fwd":
            s["res"] = _randn(g, (T, H), dt) if case["residual"] else None
        else:
            s["dy"] = _randn(g, (T, H), dt)
    return s


# ------------------------------------------------------------------ plain forms
def _act(name, z):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _expert_of_row(s):
    """Each row's expert, and its place in a [E, most] array of padded groups."""
    off = s["offsets"].long()
    r = torch.arange(s["M"], device="cuda")
    e = torch.searchsorted(off, r, right=True) - 1
    return e, e * s["most"] + r - off[e]


def _padded(s, at, t):
    p = t.new_zeros(s["E"] * s["most"], t.shape[1])
    p[at] = t
    return p.view(s["E"], s["most"], t.shape[1])


def _linear_fwd(s):
    dt = DTYPES[s["dtype"]]
    x, w = s["x"].float(), s["w"].float()
    if s["E"]:
        e, at = _expert_of_row(s)
        z = torch.bmm(_padded(s, at, x), w.transpose(1, 2)).flatten(0, 1)[at]
        z = z + s["bias_t"].float()[e] if s["bias"] else z
    else:
        z = x @ w.t()
        z = z + s["bias_t"].float() if s["bias"] else z
    y = _act(s["act"], z)
    y = y + s["res"].float() if s["residual"] else y
    return {"y": y.to(dt), "z": z.to(dt)} if s["keep"] else {"y": y.to(dt)}


def _linear_bwd(s):
    dt = DTYPES[s["dtype"]]
    x, w = s["x"].float(), s["w"].float()
    dz = s["dy"].float() * _act_grad(s["act"], s["z"].float())
    if s["E"]:
        e, at = _expert_of_row(s)
        dzp = _padded(s, at, dz)
        dx = torch.bmm(dzp, w).flatten(0, 1)[at]
        dw = torch.bmm(dzp.transpose(1, 2), _padded(s, at, x))
        db = dzp.sum(1)
    else:
        dx, dw, db = dz @ w, dz.t() @ x, dz.sum(0)
    out = {"dx": dx.to(dt), "dw": dw.to(dt)}
    if s["bias"]:
        out["db"] = db.to(dt)
    return out


def _plain(s):
    if s["op"] == "linear_fwd":
        return _linear_fwd(s)
    if s["op"] == "linear_bwd":
        return _linear_bwd(s)
    dt, T, H, k, p = DTYPES[s["dtype"]], s["T"], s["H"], s["k"], s["sched"]
    row, slot, w = p["row_of_slot"].long(), p["slot_of_row"].long(), p["topk_w"]
    if s["op"] == "permute_fwd":
        return s["x"][slot // k]
    if s["op"] == "permute_bwd":
        return s["dxs"].float()[row].view(T, k, H).sum(1).to(dt)
    o = s["o"].float()[row].view(T, k, H)
    if s["op"] == "unpermute_fwd":
        y = (o * w.unsqueeze(2)).sum(1)
        return (y + s["res"].float() if s["residual"] else y).to(dt)
    dy = s["dy"].float()
    dw = (o * dy.unsqueeze(1)).sum(2)
    dl = torch.zeros(T, s["E"], device=dy.device)
    dl.scatter_(1, p["topk_idx"].long(), w * (dw - (w * dw).sum(1, keepdim=True)))
    return {"do": (w.flatten()[slot].unsqueeze(1) * dy[slot // k]).to(dt), "dw": dw, "dl": dl}


# ------------------------------------------------------------------ the package's calls
def _own_linear(s):
    from mixture_experts_layer_dispatch_amd import binding as B

    if "lc" not in s:
        s["lc"] = B.LinearConfig(M=s["M"], N=s["N"], K=s["K"], E=s["E"], dtype=DTYPES[s["dtype"]], act=s["act"])
        s["ws"] = B.alloc_linear_workspace(s["lc"])
    lc, x, w = s["lc"], s["x"], s["w"]
    if s["op"] == "linear_fwd":
        y = x.new_empty(s["M"], s["N"])
        z = torch.empty_like(y) if s["keep"] else None
        B.moe_linear_forward(lc, x, w, y, s["ws"], bias=s["bias_t"], residual=s["res"], z=z, offsets=s["offsets"])
        return {"y": y, "z": z} if s["keep"] else {"y": y}
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    db = torch.empty_like(s["bias_t"]) if s["bias"] else None
    B.moe_linear_backward(lc, x, w, s["z"] if s["act"] != "none" else None, s["dy"], s["ws"], dx=dx, dw=dw, db=db,
                          offsets=s["offsets"])
    return {"dx": dx, "dw": dw, "db": db} if s["bias"] else {"dx": dx, "dw": dw}


def _own(s):
    from mixture_experts_layer_dispatch_amd import binding as B

    if s["op"].startswith("linear"):
        return _own_linear(s)
    if "cfg" not in s:
        s["cfg"] = B.Config(T=s["T"], H=s["H"], I=128, E=s["E"], k=s["k"])
        s["ws"] = B.alloc_error_word()
    cfg, sched, ws = s["cfg"], s["sched"], s["ws"]
    if s["op"] == "permute_fwd":
        xs = s["x"].new_empty(cfg.S, cfg.H)
        B.moe_permute_forward(cfg, sched, s["x"], xs, ws)
        return xs
    if s["op"] == "permute_bwd":
        dx = s["dxs"].new_empty(cfg.T, cfg.H)
        B.moe_permute_backward(cfg, sched, s["dxs"], dx, ws)
        return dx
    if s["op"] == "unpermute_fwd":
        y = s["o"].new_empty(cfg.T, cfg.H)
        B.moe_unpermute_forward(cfg, sched, s["o"], y, ws, residual=s["res"])
        return y
    do = torch.empty_like(s["o"])
    dw = torch.empty(cfg.T, cfg.k, device=do.device)
    dl = torch.empty(cfg.T, cfg.E, device=do.device)
    B.moe_unpermute_backward(cfg, sched, s["o"], s["dy"], do, dw, ws, d_logits=dl)
    return {"do": do, "dw": dw, "dl": dl}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("linear"):
        M, N, K, E = case["M"], case["N"], case["K"], case["E"]
        off = s["offsets"].tolist() if E else [0, M]
        f64 = dict(dtype=torch.float64, device="cuda")
        fwd = case["op"] == "linear_fwd"
        if fwd:
            y, z = torch.empty(M, N, **f64), torch.empty(M, N, **f64)
        else:
            dx, dw, db = torch.empty(M, K, **f64), torch.zeros(max(E, 1), N, K, **f64), torch.zeros(max(E, 1), N, **f64)
        for e in range(max(E, 1)):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            we = (s["w"][e] if E else s["w"]).double()
            xe = s["x"][a:b].double()
            if fwd:
                ze = torch.mm(xe, we.t())
                if case["bias"]:
                    ze += (s["bias_t"][e] if E else s["bias_t"]).double()
                z[a:b] = ze
                y[a:b] = _exact_act(case["act"], ze)[0]
                if case["residual"]:
                    y[a:b] += s["res"][a:b].double()
            else:
                dze = s["dy"][a:b].double() * _exact_act(case["act"], s["z"][a:b].double())[1]
                dx[a:b] = torch.mm(dze, we)
                dw[e] = torch.mm(dze.t(), xe)
                db[e] = dze.sum(0)
        if fwd:
            return {"y": y, "z": z} if case["keep"] else {"y": y}
        dw, db = (dw, db) if E else (dw[0], db[0])
        return {"dx": dx, "dw": dw, "db": db} if case["bias"] else {"dx": dx, "dw": dw}
    T, H, k, p = case["T"], case["H"], case["k"], s["sched"]
    if case["op"] == "permute_fwd":
        out = torch.empty(T * k, H, dtype=torch.float64, device="cuda")
        for j in range(k):
            out[p["row_of_slot"].view(T, k)[:, j].long()] = s["x"].double()
        return out
    rows = p["row_of_slot"].view(T, k).long()
    if case["op"] == "permute_bwd":
        dx = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for j in range(k):
            dx += s["dxs"][rows[:, j]].double()
        return dx
    w = p["topk_w"].double()
    if case["op"] == "unpermute_fwd":
        y = s["res"].double() if case["residual"] else torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for j in range(k):
            y += w[:, j:j + 1] * s["o"][rows[:, j]].double()
        return y
    dy = s["dy"].double()
    do = torch.empty(T * k, H, dtype=torch.float64, device="cuda")
    dw = torch.empty(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        do[rows[:, j]] = w[:, j:j + 1] * dy
        dw[:, j] = (s["o"][rows[:, j]].double() * dy).sum(1)
    # the softmax over the chosen logits: its Jacobian is diag(w) - w w^T
    jac = torch.diag_embed(w) - w.unsqueeze(2) * w.unsqueeze(1)
    dl = torch.zeros(T, case["E"], dtype=torch.float64, device="cuda")
    dl[torch.arange(T, device="cuda").unsqueeze(1), p["topk_idx"].long()] = (jac * dw.unsqueeze(1)).sum(2)
    return {"do": do, "dw": dw, "dl": dl}


def _exact_act(name, z):
    """(act(z), act'(z)) in 64 bits."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if name == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    # gelu_tanh: (1 + tanh u) / 2 = sigmoid(2u)
    u2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    p = torch.sigmoid(u2)
    return z * p, p + z * p * (1 - p) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
