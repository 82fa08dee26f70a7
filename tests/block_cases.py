"""Helpers of the building blocks' GPU tests: schedules, inputs and the
elementwise error bounds.

A value stored in a type is off by at most half a step, eps / 2 relative
(U[dtype]), or half the smallest subnormal.  An fp32 sum of n products is off
by at most n steps of 2^-23 of the sum of their magnitudes (each addition
rounds or truncates once, and no partial sum is larger than that sum).  The
fp32 activations and their derivatives are off by at most 2^-18 of
max(|z|, 1): a few roundings, and an exponential, error function or reciprocal
with errors of a few units in the last place of arguments below 2^4 (beyond
them the functions are 0, 1 or z).
"""
from __future__ import annotations

import numpy as np
import torch

from mixture_experts_layer_dispatch_amd import binding as B

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
U = {t: torch.finfo(t).eps / 2 for t in (BF, FP, F32)}
TINY = {t: float(torch.finfo(t).smallest_normal) * torch.finfo(t).eps for t in (BF, FP, F32)}
STEP = 2.0 ** -23
ACT_ERR = 2.0 ** -18
ACT_SLOPE = 1.2           # no activation here has a steeper slope (gelu: 1.129)


def n64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def randn(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def assert_within(name, got, ref, tol):
    got, ref, tol = n64(got), np.asarray(ref), np.broadcast_to(np.asarray(tol), np.shape(ref))
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), f"{name}: not finite"
    over = np.abs(got - ref) - tol
    if got.size:
        i = np.unravel_index(np.argmax(over), over.shape)
        assert over[i] <= 0, f"{name}{list(i)}: {got[i]!r}, expected {ref[i]!r} +- {tol[i]:.3e}"


def sum_err(n, mag):
    return (n + 2) * STEP * mag


def schedule(seed, T, E, k, H, macrobatch=0, skew=0.0):
    """A Config, its schedule from the framework's own routing of seeded logits, and the workspace."""
    cfg = B.Config(T=T, H=H, I=128, E=E, k=k, macrobatch=macrobatch)
    g = gen(seed)
    logits = torch.randn(T, E, generator=g, device="cuda")
    if skew:
        logits -= skew * torch.arange(E, device="cuda")
    ws = B.alloc_workspace(cfg)
    sched = B.alloc_schedule(cfg)
    B.moe_schedule(cfg, logits, sched, ws)
    return cfg, sched, ws


def group_offsets(counts):
    return torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device="cuda")
