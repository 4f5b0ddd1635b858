"""fp64 oracle of the selective mixer and of the residual pre-norm: the definitions, position by
position, in plain torch on the CPU.  Gradients are autograd's through these definitions (pinned
to differences in the tests).  Shares no code with the library.

Shapes as in ``include/ida.h``: x [B,N,H,d], b and c [B,N,G,M], dt [B,N,H], states [B,H,M,d].
"""
from __future__ import annotations

import torch


def conv(x, w, bias, state=None):
    """(out [B,N,C], last W-1 raw rows): SiLU of the causal depthwise convolution."""
    B, N, C = x.shape
    W = w.shape[1]
    head = torch.zeros(B, W - 1, C, dtype=x.dtype) if state is None else state
    rows = torch.cat([head, x], dim=1)
    pre = bias + sum(w[:, j] * rows[:, j:j + N] for j in range(W))
    return pre / (1 + torch.exp(-pre)), rows[:, N:]


def step_size(dt, dt_bias):
    z = dt + dt_bias
    return torch.where(z > 0, z + torch.log1p(torch.exp(-z.abs())), torch.log1p(torch.exp(-z.abs())))


def scan(x, b, c, dt, a_log, dt_bias, D, state=None):
    """(y [B,N,H,d], last state): the recurrence as it is written."""
    B, N, H, d = x.shape
    rep = H // b.shape[2]
    bh, ch = b.repeat_interleave(rep, 2), c.repeat_interleave(rep, 2)
    delta = step_size(dt, dt_bias)
    a = torch.exp(-torch.exp(a_log) * delta)
    X = torch.zeros(B, H, b.shape[3], d, dtype=x.dtype) if state is None else state
    ys = []
    for t in range(N):
        X = a[:, t, :, None, None] * X + delta[:, t, :, None, None] * bh[:, t, :, :, None] * x[:, t, :, None, :]
        ys.append((ch[:, t, :, :, None] * X).sum(2) + D[:, None] * x[:, t])
    return (torch.stack(ys, 1) if ys else x.clone()), X


def step(xbc, dt, p, conv_state, state, groups):
    """(y [B,H,d], conv state, state) of one position."""
    B, H, M, d = state.shape
    out, tail = conv(xbc[:, None], p["conv_w"], p["conv_b"], conv_state)
    x, b, c = out.split([H * d, groups * M, groups * M], dim=-1)
    y, X = scan(x.reshape(B, 1, H, d), b.reshape(B, 1, groups, M), c.reshape(B, 1, groups, M), dt[:, None],
                p["a_log"], p["dt_bias"], p["D"], state)
    return y[:, 0], tail, X


def rmsnorm(r, w, eps):
    return r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * w


def grads(fn, leaves, dout):
    """Gradients of sum(fn(*leaves) * dout)."""
    leaves = [t.detach().clone().requires_grad_() for t in leaves]
    return torch.autograd.grad((fn(*leaves) * dout).sum(), leaves)


def scan_parts(x, b, c, delta, log_a, D):
    """The scan from a zero state with the step sizes and the log decays as inputs of their own."""
    N, rep = x.shape[1], x.shape[2] // b.shape[2]
    bh, ch = b.repeat_interleave(rep, 2), c.repeat_interleave(rep, 2)
    a = torch.exp(log_a)
    X, ys = torch.zeros(x.shape[0], x.shape[2], b.shape[3], x.shape[3], dtype=x.dtype), []
    for t in range(N):
        X = a[:, t, :, None, None] * X + delta[:, t, :, None, None] * bh[:, t, :, :, None] * x[:, t, :, None, :]
        ys.append((ch[:, t, :, :, None] * X).sum(2) + D[:, None] * x[:, t])
    return torch.stack(ys, 1)


def scan_grad_sizes(x, b, c, dt, a_log, dt_bias, D, dy, block=64):
    """The sums of absolute terms behind each gradient of the scan (x, b, c, dt, a_log, dt_bias, D),
    which rounding errors are measured by.  The gradient of log a_t is taken as a running sum, from
    the end of a block of positions on, of c_u^T X_u dy_u - D_u b_u^T Z_u x_u: beside its own
    terms, the absolute terms of those products at u >= t of t's block stand behind it."""
    z = dt + dt_bias
    delta, rate = step_size(dt, dt_bias), torch.exp(a_log)
    gx, gb, gc, gdelta, glog, gD = grads(scan_parts, [x.abs(), b.abs(), c.abs(), delta, -rate * delta, D.abs()],
                                         dy.abs())
    pairs = (scan(x.abs(), b.abs(), c.abs(), dt, a_log, dt_bias, D.abs())[0] * dy.abs()).sum(-1) + (gx * x.abs()).sum(-1)
    for t0 in range(0, x.shape[1], block):
        glog[:, t0:t0 + block] += pairs[:, t0:t0 + block].flip(1).cumsum(1).flip(1)
    gdt = (gdelta + rate * glog) * torch.sigmoid(z)
    return gx, gb, gc, gdt, (rate * delta * glog).sum((0, 1)), gdt.sum((0, 1)), gD
