"""Refusals of routing with scores, norm and linear with 4-bit weights, on the
host: at the C entry points one wrong argument at a time (every other buffer has
an address of its own, never dereferenced), and the binding's checks of tensors.
Without a GPU a call that passes its checks ends with
MOE_ERR_UNSUPPORTED_DEVICE; with one the C calls are not made, since only the
refused ones would be safe."""
import ctypes

import pytest
import torch

from mixture_experts_layer_dispatch_amd import binding as B

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="calls that pass the checks would run")
PASSES, BAD, WS = B.MOE_ERR_UNSUPPORTED_DEVICE, B.MOE_ERR_INVALID_ARG, B.MOE_ERR_WORKSPACE
NAMES = ["logits", "bias", "topk_idx", "topk_w", "scores", "dw", "d_scores", "d_logits", "x", "residual", "gamma",
         "beta", "y", "total", "mean", "rstd", "dy", "d_total", "dx", "dgamma", "dbeta", "offsets", "codes", "scales",
         "zeros", "w", "counts", "sched_offsets", "mini_counts", "row_of_slot", "slot_of_row", "ws"]
ADDR = {n: (i + 1) << 24 for i, n in enumerate(NAMES)}
TABLE = ["topk_idx", "topk_w", "counts", "sched_offsets", "mini_counts", "row_of_slot", "slot_of_row"]
CFG = dict(T=8, H=128, I=128, E=12, k=2)
ROUTE = dict(score=0, n_group=4, topk_group=2, group_top=2, renorm=1, scale=1.0)
NORM = dict(M=16, H=256, kind=0, dtype=0, params=0, eps=1e-5)
W4 = dict(M=16, N=128, K=256, E=4, group=64, dtype=0, act=0, flags=0)

# buffers in the order of the arguments, those that may be missing, bytes of alignment that are not 16
CALLS = {"moe_route_forward": ["logits", "bias", "topk_idx", "topk_w", "scores"],
         "moe_route_backward": ["logits", "topk_idx", "dw", "d_scores", "d_logits"],
         "moe_schedule_from_topk": TABLE,
         "moe_norm_forward": ["x", "residual", "gamma", "beta", "y", "total", "mean", "rstd"],
         "moe_norm_backward": ["x", "gamma", "mean", "rstd", "dy", "d_total", "dx", "dgamma", "dbeta"],
         "moe_linear_w4_forward": ["offsets", "x", "codes", "scales", "zeros", "bias", "residual", "y"],
         "moe_linear_w4_quantize": ["w", "codes", "scales", "zeros"]}
OPTIONAL = {("moe_route_forward", "bias"), ("moe_route_forward", "scores"), ("moe_route_backward", "d_scores"),
            ("moe_norm_forward", "beta"), ("moe_norm_forward", "mean"), ("moe_norm_forward", "rstd"),
            ("moe_norm_backward", "d_total"), ("moe_norm_backward", "dgamma"), ("moe_norm_backward", "dbeta"),
            ("moe_linear_w4_forward", "zeros"), ("moe_linear_w4_forward", "bias"),
            ("moe_linear_w4_forward", "residual"), ("moe_linear_w4_quantize", "zeros")}
FOUR = {"logits", "topk_idx", "topk_w", "scores", "dw", "d_scores", "d_logits", "mean", "rstd", "offsets", *TABLE}
OUTPUTS = {"moe_route_forward": ["topk_idx", "topk_w", "scores"], "moe_route_backward": ["d_logits"],
           "moe_schedule_from_topk": TABLE, "moe_norm_forward": ["y", "total", "mean", "rstd"],
           "moe_norm_backward": ["dx", "dgamma", "dbeta"], "moe_linear_w4_forward": ["y"],
           "moe_linear_w4_quantize": ["codes", "scales", "zeros"]}
SAME = {("moe_norm_forward", "total", "x"), ("moe_norm_forward", "total", "residual"),
        ("moe_norm_backward", "dx", "dy"), ("moe_norm_backward", "dx", "d_total"),
        ("moe_linear_w4_forward", "y", "residual")}


def call(name, change=None, ws_bytes=1 << 40, cfg=True, second=True, **addr):
    """Status of the call with its configs changed and the named addresses replaced (None: null)."""
    a, change, L = {**ADDR, **addr}, change or {}, B.lib()
    pick = lambda base: {k: change.get(k, v) for k, v in base.items()}  # noqa: E731
    b = [a[n] for n in CALLS[name]]
    if name.startswith(("moe_route", "moe_schedule")):
        c = B.Config(**pick(CFG)).c() if cfg else None
        r = B.moe_route_config(*pick(ROUTE).values()) if second else None
        if name == "moe_schedule_from_topk":
            return L.moe_schedule_from_topk(c, B.moe_sched(*b) if second else None, a["ws"], ws_bytes, None)
        s = B.moe_sched(topk_idx=a["topk_idx"], topk_w=a["topk_w"] if name == "moe_route_forward" else None)
        if name == "moe_route_forward":
            return L.moe_route_forward(c, r, a["logits"], a["bias"], s, a["scores"], None)
        return L.moe_route_backward(c, r, a["logits"], s, a["dw"], a["d_scores"], a["d_logits"], a["ws"], ws_bytes, None)
    if name.startswith("moe_norm"):
        c = B.moe_norm_config(*pick(NORM).values()) if cfg else None
        tail = [a["ws"], ws_bytes] if name == "moe_norm_backward" else []
        return getattr(L, name)(c, *b, *tail, None)
    c = B.moe_linear_w4_config(*pick(W4).values()) if cfg else None
    tail = [a["ws"], ws_bytes] if name == "moe_linear_w4_forward" else []
    return getattr(L, name)(c, *b, *tail, None)


EACH = [(c, n) for c, names in CALLS.items() for n in names]


@no_gpu
def test_the_calls_pass_as_they_are():
    for name in CALLS:
        assert call(name) == PASSES, name
        assert call(name, cfg=False) == BAD
    for name, n in OPTIONAL:
        assert call(name, **{n: None}) == PASSES, (name, n)
    for name, out, other in SAME:
        assert call(name, **{out: ADDR[other]}) == PASSES
    assert call("moe_norm_forward", residual=None, total=None) == PASSES
    assert call("moe_norm_backward", dx=None, d_total=None) == PASSES
    assert call("moe_linear_w4_forward", {"E": 0}, offsets=None) == PASSES
    assert call("moe_norm_forward", {"kind": 1}, beta=None, mean=None) == PASSES
    assert call("moe_norm_backward", {"kind": 1}, mean=None, dbeta=None) == PASSES
    for name in ("moe_route_forward", "moe_route_backward", "moe_schedule_from_topk"):
        assert call(name, second=False) == BAD


@no_gpu
@pytest.mark.parametrize("name,arg", [p for p in EACH if p not in OPTIONAL and p != ("moe_norm_backward", "dx")])
def test_a_buffer_that_is_missing(name, arg):
    assert call(name, **{arg: None}) == BAD


@no_gpu
@pytest.mark.parametrize("name,arg", EACH)
def test_a_buffer_that_is_not_aligned(name, arg):
    four = arg in FOUR or (name, arg) == ("moe_route_forward", "bias")
    assert call(name, **{arg: ADDR[arg] + (2 if four else 8)}) == BAD
    if four:
        assert call(name, **{arg: ADDR[arg] + 4}) == PASSES


@no_gpu
@pytest.mark.parametrize("name,out,other", [(c, o, n) for c, outs in OUTPUTS.items() for o in outs for n in CALLS[c]
                                            if o != n and (c, o, n) not in SAME])
def test_an_output_is_no_other_buffer(name, out, other):
    assert call(name, **{out: ADDR[other]}) == BAD


@no_gpu
@pytest.mark.parametrize("name", ["moe_route_backward", "moe_schedule_from_topk", "moe_norm_backward",
                                  "moe_linear_w4_forward"])
def test_workspaces(name):
    assert call(name, ws=None) == WS
    assert call(name, ws=ADDR["ws"] + 128) == WS
    assert call(name, ws_bytes=255) == WS


@no_gpu
def test_what_belongs_together():
    f, b = "moe_norm_forward", "moe_norm_backward"
    assert call(f, residual=None) == BAD and call(f, total=None) == BAD
    for change in (dict(beta=None), dict(mean=None), {}):
        assert call(f, {"kind": 1}, **change) == BAD
    for change in (dict(mean=None), dict(dbeta=None)):
        assert call(b, {"kind": 1}, **change) == BAD
    assert call(b, dx=None) == BAD                        # d_total without dx
    assert call(b, dx=None, d_total=None, dgamma=None, dbeta=None) == BAD
    assert call("moe_linear_w4_forward", {"E": 0}) == BAD


@no_gpu
@pytest.mark.parametrize("change", [dict(score=-1), dict(score=2), dict(n_group=0), dict(n_group=5), dict(n_group=-4),
                                    dict(topk_group=0), dict(topk_group=5), dict(group_top=0), dict(group_top=3),
                                    dict(n_group=12, topk_group=4), dict(renorm=2), dict(renorm=-1),
                                    dict(k=4, topk_group=1), dict(scale=float("nan")), dict(scale=float("inf")),
                                    dict(E=130, n_group=65, topk_group=65, group_top=1), dict(E=1025, n_group=1, topk_group=1),
                                    dict(T=0), dict(k=0), dict(E=0), dict(H=100)])
def test_route_configs(change):
    assert call("moe_route_forward", change) == BAD
    assert call("moe_route_backward", change) == BAD


@no_gpu
def test_route_configs_at_their_ends():
    for change in (dict(E=128, n_group=64, topk_group=64), dict(n_group=12, topk_group=12, group_top=1), dict(scale=0.0),
                   dict(scale=-2.0), dict(k=3, topk_group=1), dict(n_group=1, topk_group=1, k=12), dict(renorm=0)):
        assert call("moe_route_forward", change) == PASSES, change


NORM_BAD = [dict(M=0), dict(M=(1 << 24) + 1), dict(H=0), dict(H=4), dict(H=12), dict(H=65544), dict(kind=2),
            dict(kind=-1), dict(dtype=3), dict(dtype=-1), dict(params=1), dict(dtype=2), dict(eps=-1e-9),
            dict(eps=float("nan")), dict(eps=float("inf"))]
W4_BAD = [dict(M=0), dict(M=(1 << 24) + 1), dict(N=0), dict(N=12), dict(N=65544), dict(K=0), dict(K=32), dict(K=96),
          dict(K=65600), dict(E=-1), dict(E=1025), dict(group=16), dict(group=96), dict(group=256), dict(dtype=2),
          dict(dtype=-1), dict(act=5), dict(act=-1), dict(flags=1)]


@pytest.mark.parametrize("change", NORM_BAD)
def test_norm_configs(change):
    n, L = ctypes.c_size_t(), B.lib()
    c = lambda **kw: B.moe_norm_config(*{**NORM, **kw}.values())  # noqa: E731
    assert L.moe_norm_workspace_size(c(), ctypes.byref(n)) == B.MOE_OK and n.value > 0
    assert L.moe_norm_workspace_size(c(dtype=2, params=2, H=65536, M=1 << 24), ctypes.byref(n)) == B.MOE_OK
    assert L.moe_norm_workspace_size(c(**change), ctypes.byref(n)) == BAD
    assert L.moe_norm_workspace_size(c(), None) == BAD and L.moe_norm_workspace_size(None, ctypes.byref(n)) == BAD
    if not torch.cuda.is_available():
        assert call("moe_norm_forward", change) == BAD
        assert call("moe_norm_backward", change) == BAD


@pytest.mark.parametrize("change", W4_BAD)
def test_w4_configs(change):
    n, L = ctypes.c_size_t(), B.lib()
    c = lambda **kw: B.moe_linear_w4_config(*{**W4, **kw}.values())  # noqa: E731
    assert L.moe_linear_w4_workspace_size(c(), ctypes.byref(n)) == B.MOE_OK and n.value >= 256
    assert L.moe_linear_w4_workspace_size(c(K=65536, group=128, E=1024, N=65536), ctypes.byref(n)) == B.MOE_OK
    assert L.moe_linear_w4_workspace_size(c(**change), ctypes.byref(n)) == BAD
    assert L.moe_linear_w4_workspace_size(c(), None) == BAD
    if not torch.cuda.is_available():
        assert call("moe_linear_w4_forward", change) == BAD
        assert call("moe_linear_w4_quantize", change) == BAD


# ------------------------------------------------------------------ the binding
BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def t(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def python_calls():
    """{name: (function of the keyword arguments, the tensors, the ones that may be None)}"""
    cfg, rc = B.Config(**CFG), B.RouteConfig()
    T, E, k = 8, 12, 2
    nc, wc = B.NormConfig(M=6, H=16), B.LinearW4Config(M=6, N=16, K=64, E=3, group=32)
    full = B.alloc_schedule(cfg, "cpu")

    def schedule(ws, **s):
        return B.moe_schedule_from_topk(cfg, s, ws)

    def route_f(topk_idx, topk_w, **kw):
        return B.moe_route_forward(cfg, rc, sched={"topk_idx": topk_idx, "topk_w": topk_w}, **kw)

    def route_b(topk_idx, **kw):
        return B.moe_route_backward(cfg, rc, sched={"topk_idx": topk_idx}, **kw)

    return {
        "route_forward": (route_f, dict(logits=t(T, E, dtype=F32), topk_idx=t(T, k, dtype=I32),
                                        topk_w=t(T, k, dtype=F32), bias=t(E, dtype=F32), scores=t(T, E, dtype=F32)),
                          ("bias", "scores")),
        "route_backward": (route_b, dict(logits=t(T, E, dtype=F32), topk_idx=t(T, k, dtype=I32),
                                         dw=t(T, k, dtype=F32), d_logits=t(T, E, dtype=F32), ws=t(256, dtype=U8),
                                         d_scores=t(T, E, dtype=F32)), ("d_scores",)),
        "schedule": (schedule, dict(ws=t(B.workspace_size(cfg), dtype=U8), **full), ()),
        "norm_forward": (lambda **kw: B.moe_norm_forward(nc, **kw),
                         dict(x=t(6, 16), gamma=t(16), y=t(6, 16), beta=t(16), residual=t(6, 16), total=t(6, 16),
                              mean=t(6, dtype=F32), rstd=t(6, dtype=F32)), ("beta", "mean", "rstd")),
        "norm_backward": (lambda **kw: B.moe_norm_backward(nc, **kw),
                          dict(x=t(6, 16), gamma=t(16), rstd=t(6, dtype=F32), dy=t(6, 16), dx=t(6, 16),
                               ws=t(B.norm_workspace_size(nc), dtype=U8), mean=t(6, dtype=F32), d_total=t(6, 16),
                               dgamma=t(16), dbeta=t(16)), ("d_total", "dgamma", "dbeta")),
        "w4_forward": (lambda **kw: B.moe_linear_w4_forward(wc, **kw),
                       dict(x=t(6, 64), codes=t(3, 16, 32, dtype=U8), scales=t(3, 2, 16), y=t(6, 16),
                            ws=t(B.linear_w4_workspace_size(wc), dtype=U8), zeros=t(3, 2, 16, dtype=U8),
                            bias=t(3, 16), residual=t(6, 16), offsets=t(4, dtype=I32)), ("zeros", "bias", "residual")),
        "w4_quantize": (lambda **kw: B.moe_linear_w4_quantize(wc, **kw),
                        dict(w=t(3, 16, 64), codes=t(3, 16, 32, dtype=U8), scales=t(3, 2, 16),
                             zeros=t(3, 2, 16, dtype=U8)), ("zeros",)),
    }


@pytest.mark.parametrize("name", list(python_calls()))
def test_the_binding_checks_every_tensor(name):
    f, args, optional = python_calls()[name]
    with pytest.raises(ValueError, match="on the GPU"):               # all is right but the device
        f(**args)
    for n in optional:
        with pytest.raises(ValueError, match="on the GPU"):
            f(**{**args, n: None})
    for n, v in args.items():
        label = "workspace" if n == "ws" else n
        wrong = [(None, "missing|given if and only if|only with dx")] if n not in optional else []
        wrong += [("no tensor", "expected"), (v.double(), "dtype")]
        if n == "ws":
            wrong.append((v[:-1].clone(), "bytes"))
        else:
            wrong.append((torch.zeros(*v.shape[:-1], v.shape[-1] + 1, dtype=v.dtype), "shape"))
            if v.dim() > 1 and v.shape[0] > 1 and v.shape[-1] > 1:
                wrong.append((torch.zeros(*v.shape[:-2], v.shape[-1], v.shape[-2], dtype=v.dtype).transpose(-1, -2),
                              "contiguous"))
        for w, why in wrong:
            if n == "dx" and w is None:
                continue                                               # (dx may be missing, without d_total)
            with pytest.raises(ValueError, match=why) as e:
                f(**{**args, n: w})
            assert label in str(e.value), (name, n, why, str(e.value))


def test_the_binding_checks_configs():
    for kw, why in ((dict(score="tanh"), "score"), (dict(n_group=1 << 32), "n_group")):
        with pytest.raises(ValueError, match=why):
            B.RouteConfig(**kw).checked
    for kw, why in ((dict(kind="group"), "kind"), (dict(dtype=torch.float64), "dtype"), (dict(params=torch.float16), "params"),
                    (dict(M=(1 << 32) + 8), "M"), (dict(H=(1 << 32) + 8), "H")):
        with pytest.raises(ValueError, match=why):
            B.NormConfig(**{**dict(M=8, H=8), **kw}).checked
    for kw, why in ((dict(act="tanh"), "act"), (dict(dtype=F32), "dtype"), (dict(group=(1 << 32) + 32), "group"),
                    (dict(K=(1 << 32) + 64), "K")):
        with pytest.raises(ValueError, match=why):
            B.LinearW4Config(**{**dict(M=8, N=8, K=64, group=32), **kw}).checked
    for bad in (B.NormConfig(M=8, H=12), B.LinearW4Config(M=8, N=8, K=96)):
        with pytest.raises(B.MoEError, match="invalid argument"):
            bad.checked


def test_the_binding_checks_what_belongs_together():
    calls = python_calls()
    f, a, _ = calls["norm_forward"]
    rms = B.NormConfig(M=6, H=16, kind="rms")
    with pytest.raises(ValueError, match="total"):
        f(**{**a, "residual": None})
    with pytest.raises(ValueError, match="rms"):
        B.moe_norm_forward(rms, **a)
    f, a, _ = calls["norm_backward"]
    with pytest.raises(ValueError, match="mean"):
        B.moe_norm_backward(rms, **a)
    with pytest.raises(ValueError, match="dbeta"):
        B.moe_norm_backward(rms, **{**a, "mean": None})
    with pytest.raises(ValueError, match="d_total"):
        f(**{**a, "dx": None})
    with pytest.raises(ValueError, match="at least one"):
        f(**{**a, "dx": None, "dgamma": None, "dbeta": None})
    f, a, _ = calls["w4_forward"]
    with pytest.raises(ValueError, match="offsets"):
        f(**{**a, "offsets": None})
