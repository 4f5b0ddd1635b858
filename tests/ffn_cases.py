"""Inputs, 64-bit references and error bounds shared by the tests of the feed-forward block and of the
products in 8 bits.

Bounds are elementwise, from the roundings that a value passes: HALF for each rounding to the type, STEP
for the block's activation, and for a sum of n products a multiple
of sum |a| |b|: the tensor cores add 16 products (32 in 8 bits) at a time and round the running sum towards zero,
each by less than 2^-23 of a partial sum, and align the products of a step to its largest with 2^-24 at least."""
from __future__ import annotations

import torch

from tests.ssm_cases import DT, HALF, gen

# The activation's own error.  bf16 (and 8 bits): the exponential of a rounded x log2 e, off by |x| 2^-24 of its value and
# 2^-22, |x| < 88 (where e^-x ends), the reciprocal's 2^-23 and three products: below 2^-17.  fp32: expf within two
# units, a division and two products: below 2^-20.
STEP = {"bf16": 2.0 ** -17, "f32": 2.0 ** -20}
# What lies below the types' least normal numbers (2^-126 in either) may be lost: the gate's sigmoid s, where 1 / s passes
# 2^126 (its reciprocal is 0 from there on: an error of 2^-126 at most, times what it multiplies), a rounded value
# and a product in a sum (2^-126 at most each).
TINY = 2.0 ** -126
E4M3 = torch.float8_e4m3fn


def sum_err(n, dtype):
    """Error of a sum of n products relative to the sum of their magnitudes."""
    if dtype == "f32":
        # 32 steps of 16 in TMEM (2^-23 each, and 16 alignments of 2^-24 in each), then fp32 additions; the parts'
        # products that are left out are below 2^-24 three times over, and there are six passes
        return 32 * 2.0 ** -23 + 16 * 2.0 ** -24 + (6 * (n / 512 + 1) + 3) * 2.0 ** -24
    return (n / 16 + 1) * 2.0 ** -23 + 16 * 2.0 ** -24


def weights(D, F, dtype, seed):
    g = gen(seed)
    return [(torch.randn(*s, generator=g) * s[1] ** -0.5).to(DT[dtype]) for s in ((F, D), (F, D), (D, F))]


def rows(T, D, dtype, seed):
    return torch.randn(T, D, generator=gen(seed)).to(DT[dtype])


def forward_ref(x, wg, wu, wd, dtype):
    """{name: (value, bound)} of out and acts."""
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    half, cd = HALF[dtype], sum_err(x.shape[1], dtype)
    g, u = x @ wg.t(), x @ wu.t()
    eg, eu = cd * (x.abs() @ wg.abs().t()), cd * (x.abs() @ wu.abs().t())
    s = g * torch.sigmoid(g)
    h = s * u
    eh = 1.01 * (1.1 * u.abs() * eg + s.abs() * eu) + (STEP[dtype] + half) * h.abs() + TINY * (1 + (g * u).abs())  # |silu'| < 1.1
    out = h @ wd.t()
    eo = eh @ wd.abs().t() + sum_err(wg.shape[0], dtype) * (h.abs() @ wd.abs().t()) + half * out.abs() + TINY * (1 + wg.shape[0])
    return {"out": (out, eo), "g": (g, eg + half * g.abs()), "u": (u, eu + half * u.abs()), "h": (h, eh)}


def backward_ref(x, wg, wu, wd, acts, dy, dtype):
    """{name: (value, bound)} of the gradients."""
    x, wg, wu, wd, dy = (t.double() for t in (x, wg, wu, wd, dy))
    g, u, h = acts.double().unbind()
    F, T, half = wg.shape[0], x.shape[0], HALF[dtype]
    s = torch.sigmoid(g)
    silu, dsilu = g * s, s * (1 + g * (1 - s))
    dh = dy @ wd
    edh = sum_err(wd.shape[0], dtype) * (dy.abs() @ wd.abs())
    du, dg = dh * silu, dh * u * dsilu
    edu = 1.01 * edh * silu.abs() + (half + STEP[dtype]) * du.abs() + TINY * (1 + (dh * g).abs())
    edg = 1.01 * edh * (u * dsilu).abs() + half * dg.abs() + STEP[dtype] * (dh * u).abs() * (s + (g * s * (1 - s)).abs()) + TINY * (1 + (dh * u).abs() * (1 + g.abs()))
    c2f, ct = sum_err(2 * F, dtype), sum_err(T, dtype)
    dx = dg @ wg + du @ wu
    edx = edg @ wg.abs() + edu @ wu.abs() + c2f * (dg.abs() @ wg.abs() + du.abs() @ wu.abs()) + half * dx.abs() + TINY * (1 + 2 * F)
    r = {"x": (dx, edx)}
    for name, a, ea, b in (("w_gate", dg, edg, x), ("w_up", du, edu, x), ("w_down", dy, None, h)):
        v = a.t() @ b
        e = ct * (a.abs().t() @ b.abs()) + half * v.abs() + TINY * (1 + T)
        r[name] = (v, e if ea is None else e + ea.t() @ b.abs())
    return r


def quantised(x, block_rows):
    """(q, scale) in fp32 as the definition has them: q in e4m3, a scale for 128 channels of `block_rows` rows."""
    T, K = x.shape
    n, k = -(-T // block_rows), -(-K // 128)
    full = torch.zeros(n * block_rows, k * 128)
    full[:T, :K] = x.float()
    v = full.view(n, block_rows, k, 128)
    top = v.abs().amax((1, 3))
    scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    q = (v / scale[:, None, :, None]).clamp(-448, 448).reshape(n * block_rows, k * 128)[:T, :K]
    return q.to(E4M3).contiguous(), scale


def values(q, scale, block_rows):
    """What q and its scales stand for, in 64 bits."""
    T, K = q.shape
    return q.float().double() * scale.double().repeat_interleave(block_rows, 0)[:T].repeat_interleave(128, 1)[:, :K]


def product_err(K):
    """Error of a product in 8 bits relative to the sum of magnitudes: in a block four steps towards zero and the alignment
    of 32 products; then a product of scales (2^-24) and a fused addition for each block."""
    return 4 * 2.0 ** -23 + 32 * 2.0 ** -24 + (1 + -(-K // 128)) * 2.0 ** -24


def product_ref(a, b):
    """(value, bound) of a b^T for operands in 64 bits, before the output's rounding."""
    v = a @ b.t()
    return v, product_err(a.shape[1]) * (a.abs() @ b.abs().t())


def glu_ref(a, wg, wu):
    """(h, bound) in 64 bits, before it is quantised."""
    (g, eg), (u, eu) = product_ref(a, wg), product_ref(a, wu)
    s = g * torch.sigmoid(g)
    h = s * u
    return h, 1.01 * (1.1 * u.abs() * eg + s.abs() * eu) + STEP["bf16"] * h.abs()
