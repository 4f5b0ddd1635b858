"""Inputs and error bounds shared by the tests of the selective mixer."""
from __future__ import annotations

import math

import torch

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step of the type, relative to the value
U32 = 2.0 ** -24


def gen(seed):
    return torch.Generator().manual_seed(seed)


def params(H, C, W, seed, fast=False):
    """conv_w, conv_b, a_log, dt_bias, D in float32; ``fast``: decays of e^-5 and more a position."""
    g = gen(seed)
    step = torch.exp(math.log(1e-3) + torch.rand(H, generator=g) * math.log(100.0))
    if fast:
        step = 1.0 + step
    return {"conv_w": torch.randn(C, W, generator=g) * W ** -0.5, "conv_b": torch.randn(C, generator=g) * 0.1,
            "a_log": torch.log(1 + 15 * torch.rand(H, generator=g)),
            "dt_bias": torch.log(torch.expm1(step)), "D": 1 + 0.1 * torch.randn(H, generator=g)}


def rows(B, N, C, H, dtype, seed):
    """One projected row per position: C convolved channels, H step sizes, padding to 8."""
    return torch.randn(B, N, (C + H + 7) // 8 * 8, generator=gen(seed)).to(DT[dtype])


def split(xbc, H, d, G, M):
    x, b, c = xbc.split([H * d, G * M, G * M], dim=-1)
    return x.unflatten(-1, (H, d)), b.unflatten(-1, (G, M)), c.unflatten(-1, (G, M))


def to64(p):
    return {k: v.double() for k, v in p.items()}


def cuda(p):
    return {k: v.cuda() for k, v in p.items()}


def worst(got, ref, bound):
    """max of |got - ref| / bound (0 where both are equal)."""
    err = (got.detach().cpu().double() - ref).abs()
    bound = torch.as_tensor(bound, dtype=torch.float64).expand_as(err)
    return float(torch.where(err == 0, torch.zeros_like(err), err / bound.clamp_min(1e-300)).max()) if err.numel() else 0.0
