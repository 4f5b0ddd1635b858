"""The selective state-space mixer and the pre-norm around it, as measured operators.

``listed()`` gives the measured cases and ``draw()`` more of the same ranges; ``prepare()`` makes a
case's inputs from a seed; ``run()`` makes one pass, either through the library (``own``) or in a
plain form of elementary torch operations; ``exact()`` evaluates the definition in 64 bits.

Operators (B rows of N positions, H heads of d channels, G groups of M state channels that H / G
heads share, C = H d + 2 G M convolved channels [x | b | c], W taps):

  conv      out = SiLU(bias + causal depthwise conv of width W)
  scan      D_t = softplus(dt_t + dt_bias), a_t = exp(-exp(a_log) D_t),
            X_t = a_t X_{t-1} + D_t b_t x_t^T, y_t = X_t^T c_t + D x_t
  step      one position of conv and scan together, both states updated in place
  norm      r = x + residual, out = r / sqrt(mean r^2 + eps) * w, optionally in e4m3 with a scale
            per group of channels
  *_bwd     the gradients of conv, scan and norm
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
E4M3_MAX = 448.0


# ---- cases -------------------------------------------------------------------------------

def listed():
    return [
        # the convolved channels of the 1.3B-like prompt (16 heads of 128, one group of 64)
        dict(name="conv_1p3b", op="conv", dtype="bf16", B=4, N=4096, H=16, d=128, M=64, G=1, W=4, state=False),
        # training the 125M-like layer: the convolution's gradients
        dict(name="conv_bwd_125m", op="conv_bwd", dtype="bf16", B=8, N=2048, H=12, d=64, M=64, G=1, W=4,
             state=False),
        # the 1.3B-like prompt at the training context
        dict(name="scan_1p3b", op="scan", dtype="bf16", B=4, N=4096, H=16, d=128, M=64, G=1, state=False),
        # one long prompt continued from a state and handed on to decoding
        dict(name="scan_14k_state", op="scan", dtype="bf16", B=1, N=14336, H=16, d=128, M=64, G=2, state=True),
        # a short ragged fp32 prompt, where latency counts
        dict(name="scan_tiny_f32", op="scan", dtype="f32", B=1, N=251, H=2, d=32, M=16, G=1, state=True),
        # training the 125M-like layer: the scan's gradients
        dict(name="scan_bwd_125m", op="scan_bwd", dtype="bf16", B=8, N=2048, H=12, d=64, M=64, G=1, state=False),
        # a small fp32 training step with an odd length and shared groups
        dict(name="scan_bwd_f32", op="scan_bwd", dtype="f32", B=2, N=509, H=4, d=32, M=16, G=2, state=False),
        # one token of one sequence
        dict(name="step_one", op="step", dtype="bf16", B=1, H=16, d=128, M=64, G=1, W=4),
        # one token of each of 256 sequences, the decode batch
        dict(name="step_256", op="step", dtype="bf16", B=256, H=16, d=128, M=64, G=1, W=4),
        # the pre-norm of the 1.3B-like prompt, for a projection in 8 bits
        dict(name="norm_1p3b_e4m3", op="norm", dtype="bf16", T=16384, D=2048, residual=True, group=128),
        # the pre-norm of a few decoded tokens
        dict(name="norm_decode", op="norm", dtype="bf16", T=5, D=2048, residual=True, group=0),
        # training the 125M-like layer: the pre-norm's gradients
        dict(name="norm_bwd_125m", op="norm_bwd", dtype="bf16", T=16384, D=768, residual=True, group=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["conv", "conv_bwd", "scan", "scan", "scan_bwd", "step", "norm", "norm_bwd"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    if op in ("norm", "norm_bwd"):
        D = 8 * _log(rng, 8, 512)
        T = _log(rng, 1, min(20000, 16384 * 2048 // D))
        group = 0
        if op == "norm" and rng.random() < 0.6:
            group = rng.choice([g for g in (32, 64, 128, D) if D % g == 0])
        return dict(op=op, dtype=dtype, T=T, D=D, residual=rng.random() < 0.8, group=group)
    d = rng.choice([64, 128]) if rng.random() < 0.7 else 8 * rng.randint(2, 16)
    M = rng.choice([64, 128]) if rng.random() < 0.7 else 8 * rng.randint(2, 16)
    H = _log(rng, 1, 32)
    G = rng.choice([g for g in range(1, H + 1) if H % g == 0])
    if op == "step":
        B = _log(rng, 1, max(1, min(256, 256 * 16 * 8192 // (H * d * M))))
        return dict(op=op, dtype=dtype, B=B, H=H, d=d, M=M, G=G, W=rng.randint(2, 4))
    if op in ("conv", "conv_bwd"):
        C = H * d + 2 * G * M
        most = (4 * 4096 * 2176 if op == "conv" else 8 * 2048 * 896) // C
        N = _log(rng, 1, min(14336, most))
        return dict(op=op, dtype=dtype, B=_log(rng, 1, max(1, min(64, most // N))), N=N, H=H, d=d, M=M, G=G,
                    W=rng.randint(2, 4), state=op == "conv" and rng.random() < 0.5)
    most = (4 * 4096 * 16 * 8192 if op == "scan" else 8 * 2048 * 12 * 4096) // (H * d * M)
    if dtype == "f32":
        most = max(1, most // 8)
    N = _log(rng, 1, max(1, min(14336, most)))
    return dict(op=op, dtype=dtype, B=_log(rng, 1, max(1, min(64, most // N))), N=N, H=H, d=d, M=M, G=G,
                state=op == "scan" and rng.random() < 0.5)


# ---- inputs ------------------------------------------------------------------------------

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def prepare(case, seed):
    g = _gen(seed)

    def randn(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    op, dt = case["op"], _DT[case["dtype"]]
    s = {"case": case}
    if op in ("norm", "norm_bwd"):
        T, D = case["T"], case["D"]
        s["w"] = 1.0 + randn(D, scale=0.1)
        if op == "norm":
            s["x"] = randn(T, D).to(dt)
            s["residual"] = randn(T, D, scale=2.0).to(dt) if case["residual"] else None
        else:
            s["r"] = randn(T, D, scale=2.0).to(dt)
            s["dy"] = randn(T, D).to(dt)
            s["dres"] = randn(T, D).to(dt) if case["residual"] else None
        return s
    H, d, M, G = case["H"], case["d"], case["M"], case["G"]
    C = H * d + 2 * G * M
    if "W" in case:
        W = case["W"]
        s["conv_w"] = randn(C, W, scale=W ** -0.5)
        s["conv_b"] = randn(C, scale=0.1)
    if op not in ("conv", "conv_bwd"):
        # rates 1 .. 16 and step sizes log-uniform on 1e-3 .. 1e-1 about which dt varies
        s["a_log"] = torch.log(1.0 + 15.0 * rand(H))
        step = torch.exp(math.log(1e-3) + rand(H) * (math.log(1e-1) - math.log(1e-3)))
        s["dt_bias"] = torch.log(torch.expm1(step))
        s["D"] = 1.0 + randn(H, scale=0.1)
    B = case["B"]
    row = (C + H + 7) // 8 * 8  # one projected row: the convolved channels, the step sizes, padding
    if op == "step":
        s["proj"] = randn(B, row).to(dt)
        s["tail"] = randn(B, case["W"] - 1, C).to(dt).float()
        s["state"] = randn(B, H, M, d, scale=0.3)
        return s
    N = case["N"]
    s["proj"] = randn(B, N, row).to(dt)
    if op in ("conv", "conv_bwd"):
        s["tail_in"] = randn(B, case["W"] - 1, C).to(dt).float() if case["state"] else None
        if op == "conv_bwd":
            s["dout"] = randn(B, N, C).to(dt)
        return s
    z = s["proj"][..., :C].float()
    s["xbc"] = (z * torch.sigmoid(z)).to(dt)  # what the convolution hands on
    if case["state"]:
        s["state_in"] = randn(B, H, M, d, scale=0.3)
    if op == "scan_bwd":
        s["dy"] = randn(B, N, H, d).to(dt)
    return s


def _split(xbc, case):
    H, d, M, G = case["H"], case["d"], case["M"], case["G"]
    x, b, c = xbc.split([H * d, G * M, G * M], dim=-1)
    return (x.unflatten(-1, (H, d)), b.unflatten(-1, (G, M)), c.unflatten(-1, (G, M)))


def _dt_of(s, case):
    C = case["H"] * case["d"] + 2 * case["G"] * case["M"]
    return s["proj"][..., C:C + case["H"]]


# ---- the library -------------------------------------------------------------------------

def _run_own(s):
    from linear_token_mixer_sc_gb300 import binding

    case = s["case"]
    op = case["op"]
    if op == "norm":
        out, res, q, scale = binding.ida_rmsnorm(s["x"], s["w"], residual=s["residual"], eps=EPS,
                                                 group=case["group"])
        got = {"q": q, "scale": scale} if case["group"] else {"out": out}
        if s["residual"] is not None:
            got["res"] = res
        return got
    if op == "norm_bwd":
        g = binding.ida_rmsnorm_backward(s["r"], s["w"], s["dy"], dres=s["dres"], eps=EPS)
        return {"dx": g["x"], "dw": g["w"]}
    C = case["H"] * case["d"] + 2 * case["G"] * case["M"]
    if op == "conv":
        out, tail = binding.ida_ssm_conv(s["proj"][..., :C], s["conv_w"], s["conv_b"], state_in=s["tail_in"],
                                         final_state=True)
        return {"out": out, "tail": tail}
    if op == "conv_bwd":
        g = binding.ida_ssm_conv_backward(s["proj"][..., :C], s["dout"], s["conv_w"], s["conv_b"])
        return {"dx": g["x"], "dw": g["conv_w"], "db": g["conv_b"]}
    if op == "step":
        y = binding.ida_ssm_step(s["proj"][..., :C], _dt_of(s, case), s, s["tail"], s["state"], case["G"])
        return {"y": y, "state": s["state"], "tail": s["tail"]}
    x, b, c = _split(s["xbc"], case)
    if op == "scan":
        y, state = binding.ida_ssm_scan(x, b, c, _dt_of(s, case), s, state_in=s.get("state_in"),
                                        final_state=case["state"])
        return {"y": y, "state": state} if case["state"] else {"y": y}
    g = binding.ida_ssm_scan_backward(x, b, c, _dt_of(s, case), s, s["dy"])
    return {"dx": g["x"], "db": g["b"], "dc": g["c"], "ddt": g["dt"], "da_log": g["a_log"],
            "ddt_bias": g["dt_bias"], "dD": g["D"]}


# ---- the plain forms ---------------------------------------------------------------------

def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _softplus(z):
    return torch.clamp(z, min=0) + torch.log1p(torch.exp(-torch.abs(z)))


def _windows(x, tail, W):
    """[..., N, C, W]: the W rows that end at each position; `tail` the rows before the first."""
    head = x.new_zeros(x.shape[0], W - 1, x.shape[2]) if tail is None else tail
    return torch.cat([head, x], dim=1).unfold(1, W, 1)


def _plain_scan(x, b, c, dt, a_log, dt_bias, D, state_in):
    """y [B,N,H,d] and the last state [B,H,M,d], by blocks of 64 positions; all in 32 bits but the
    sums of log decays, whose differences over long ranges need 64."""
    B, N, H, d = x.shape
    M, Q = b.shape[3], 64
    n = (N + Q - 1) // Q
    pad = n * Q - N
    rep = H // b.shape[2]
    delta = _softplus(dt + dt_bias)
    log_a = -torch.exp(a_log.double()) * delta.double()

    def blocks(v):  # [B,N,H,...] -> [B,H,n,Q,...]
        v = torch.cat([v, v.new_zeros(B, pad, *v.shape[2:])], dim=1)
        return v.unflatten(1, (n, Q)).movedim(3, 1)

    xb, bb, cb = blocks(x), blocks(b.repeat_interleave(rep, 2)), blocks(c.repeat_interleave(rep, 2))
    db, la = blocks(delta), blocks(log_a)
    cum = la.cumsum(-1)
    keep = torch.ones(Q, Q, dtype=torch.bool, device=x.device).tril()
    seg = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~keep, -math.inf)).float()
    y = ((cb @ bb.transpose(-1, -2)) * seg * db[..., None, :]) @ xb
    to_end = torch.exp(cum[..., -1:] - cum).float() * db
    local = (bb * to_end[..., None]).transpose(-1, -2) @ xb  # [B,H,n,M,d]
    start = x.new_zeros(B, H, 1, M, d) if state_in is None else state_in[:, :, None]
    total = torch.cat([cum.new_zeros(B, H, 1), cum[..., -1].cumsum(-1)], dim=-1)  # before block i
    keep = torch.ones(n + 1, n + 1, dtype=torch.bool, device=x.device).tril()
    carry = torch.exp((total[..., :, None] - total[..., None, :]).masked_fill(~keep, -math.inf)).float()
    states = (carry @ torch.cat([start, local], dim=2).flatten(3)).unflatten(-1, (M, d))
    y = y + (cb * torch.exp(cum).float()[..., None]) @ states[:, :, :-1]
    y = y.movedim(1, 3).flatten(1, 2)[:, :N] + D[:, None] * x
    return y, states[:, :, -1]


def _plain_norm(x, residual, w, dt):
    r = x.float() if residual is None else (x.float() + residual.float()).to(dt).float()
    return r, r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * w


def _run_plain(s):
    case = s["case"]
    op, dt = case["op"], _DT[case["dtype"]]
    if op == "norm":
        r, y = _plain_norm(s["x"], s["residual"], s["w"], dt)
        got = {} if s["residual"] is None else {"res": r.to(dt)}
        if case["group"]:
            yg = y.unflatten(-1, (-1, case["group"]))
            amax = yg.abs().amax(-1, keepdim=True)
            scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
            q = torch.clamp(yg / scale, -E4M3_MAX, E4M3_MAX).flatten(1)
            return {**got, "q": q.to(torch.float8_e4m3fn), "scale": scale[..., 0]}
        return {**got, "out": y.to(dt)}
    if op == "norm_bwd":
        r, dy = s["r"].float(), s["dy"].float()
        inv = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
        gw = dy * s["w"]
        dx = inv * (gw - r * (inv * inv) * (gw * r).mean(-1, keepdim=True))
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        return {"dx": dx.to(dt), "dw": (dy * r * inv).sum(0)}
    H, d, M, G = case["H"], case["d"], case["M"], case["G"]
    C = H * d + 2 * G * M
    if op == "conv":
        x = s["proj"][..., :C].float()
        win = _windows(x, s["tail_in"], case["W"])
        out = _silu((win * s["conv_w"]).sum(-1) + s["conv_b"])
        tail = torch.cat([torch.zeros_like(win[:, 0]) if s["tail_in"] is None else
                          torch.cat([torch.zeros_like(x[:, :1]), s["tail_in"]], 1).transpose(1, 2),
                          x.transpose(1, 2)], dim=-1)[..., 1 - case["W"]:].transpose(1, 2)
        return {"out": out.to(dt), "tail": tail.contiguous()}
    if op == "conv_bwd":
        x, W = s["proj"][..., :C].float(), case["W"]
        win = _windows(x, None, W)
        pre = (win * s["conv_w"]).sum(-1) + s["conv_b"]
        sig = 1.0 / (1.0 + torch.exp(-pre))
        dpre = s["dout"].float() * sig * (1.0 + pre * (1.0 - sig))
        ahead = torch.cat([dpre, dpre.new_zeros(dpre.shape[0], W - 1, C)], dim=1).unfold(1, W, 1)
        dx = (ahead * s["conv_w"].flip(-1)).sum(-1)
        return {"dx": dx.to(dt), "dw": (win * dpre[..., None]).sum((0, 1)), "db": dpre.sum((0, 1))}
    if op == "step":
        row = s["proj"][..., :C].float()
        win = torch.cat([s["tail"], row[:, None]], dim=1)  # [B,W,C]
        xbc = _silu((win * s["conv_w"].t()).sum(1) + s["conv_b"])
        x, b, c = _split(xbc, case)
        b, c = b.repeat_interleave(H // G, 1), c.repeat_interleave(H // G, 1)
        delta = _softplus(_dt_of(s, case).float() + s["dt_bias"])
        a = torch.exp(-torch.exp(s["a_log"]) * delta)
        state = a[..., None, None] * s["state"] + (delta[..., None] * b)[..., None] * x[..., None, :]
        y = (c[..., None] * state).sum(2) + s["D"][:, None] * x
        s["state"].copy_(state)
        s["tail"].copy_(win[:, 1:])
        return {"y": y.to(dt), "state": s["state"], "tail": s["tail"]}
    x, b, c = _split(s["xbc"], case)
    dtv = _dt_of(s, case)
    if op == "scan":
        y, state = _plain_scan(x.float(), b.float(), c.float(), dtv.float(), s["a_log"], s["dt_bias"], s["D"],
                               s.get("state_in"))
        return {"y": y.to(dt), "state": state.contiguous()} if case["state"] else {"y": y.to(dt)}
    leaves = [t.detach().float().requires_grad_() for t in (x, b, c, dtv, s["a_log"], s["dt_bias"], s["D"])]
    with torch.enable_grad():
        y, _ = _plain_scan(*leaves, None)
        g = torch.autograd.grad(y, leaves, s["dy"].float())
    return {"dx": g[0].to(dt), "db": g[1].to(dt), "dc": g[2].to(dt), "ddt": g[3].to(dt), "da_log": g[4],
            "ddt_bias": g[5], "dD": g[6]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op == "norm":
        T, D = case["T"], case["D"]
        rows = 1 + (2 if case["residual"] else 0)  # x, and with a residual its two rows
        out = T * D + 4 * T * D // case["group"] if case["group"] else T * D * e
        return {"bytes": T * D * e * rows + out + 4 * D, "flops": 6 * T * D}
    if op == "norm_bwd":
        T, D = case["T"], case["D"]
        return {"bytes": T * D * e * (4 if case["residual"] else 3) + 8 * D, "flops": 11 * T * D}
    B, H, d, M, G = case["B"], case["H"], case["d"], case["M"], case["G"]
    C = H * d + 2 * G * M
    if op == "step":
        W = case["W"]
        return {"bytes": 8 * B * H * M * d + 8 * B * (W - 1) * C + e * B * (C + H + H * d) + 4 * C * (W + 1) + 12 * H,
                "flops": 6 * B * H * M * d + (2 * W + 4) * B * C}
    N = case["N"]
    if op == "conv":
        W = case["W"]
        return {"bytes": 2 * e * B * N * C + 4 * B * (W - 1) * C * (2 if case["state"] else 1) + 4 * C * (W + 1),
                "flops": (2 * W + 4) * B * N * C}
    if op == "conv_bwd":
        W = case["W"]
        return {"bytes": 3 * e * B * N * C + 8 * C * (W + 1), "flops": (6 * W + 10) * B * N * C}
    # the recurrence itself: update, read-out; backwards two adjoint products and the update more
    states = (2 if case["state"] else 0) * 4 * B * H * M * d
    if op == "scan":
        return {"bytes": e * B * N * (C + H + H * d) + states + 12 * H, "flops": 5 * B * N * H * M * d}
    return {"bytes": e * B * N * (2 * (C + H) + H * d) + 24 * H, "flops": 14 * B * N * H * M * d}


# ---- the definitions in 64 bits ------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        w = s["w"].double()
        if op == "norm":
            total = s["x"].double()
            if s["residual"] is not None:
                total = total + s["residual"].double()
            r = total.to(_DT[case["dtype"]]).double()  # the stored stream is what is normalised
            y = r / (r.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w
            got = {} if s["residual"] is None else {"res": total}
            if case["group"]:
                top = y.reshape(case["T"], -1, case["group"]).abs().max(-1).values
                return {**got, "q": None, "scale": torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))}
            return {**got, "out": y}
        r, dy = s["r"].double(), s["dy"].double()
        rms = (r.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
        n = r / rms
        dn = dy * w
        dx = (dn - n * (dn * n).mean(-1, keepdim=True)) / rms
        if s["dres"] is not None:
            dx = dx + s["dres"].double()
        return {"dx": dx, "dw": (dy * n).sum(0)}
    H, d, M, G = case["H"], case["d"], case["M"], case["G"]
    C = H * d + 2 * G * M
    if "W" in case:
        w, bias, W = s["conv_w"].double(), s["conv_b"].double(), case["W"]
    if op in ("conv", "conv_bwd"):
        x = s["proj"][..., :C].double()
        N = x.shape[1]
        head = torch.zeros(x.shape[0], W - 1, C, dtype=x.dtype, device=x.device)
        if s["tail_in"] is not None:
            head = s["tail_in"].double()
        rows = torch.cat([head, x], 1)
        pre = bias + sum(w[:, j] * rows[:, j:j + N] for j in range(W))
        sig = torch.sigmoid(pre)
        if op == "conv":
            return {"out": pre * sig, "tail": rows[:, N:]}
        dpre = s["dout"].double() * (sig + pre * sig * (1 - sig))
        dx = torch.zeros_like(x)
        for j in range(W):
            k = W - 1 - j
            if k < N:
                dx[:, :N - k] += w[:, j] * dpre[:, k:]
        dw = torch.stack([(rows[:, j:j + N] * dpre).sum((0, 1)) for j in range(W)], -1)
        return {"dx": dx, "dw": dw, "db": dpre.sum((0, 1))}
    rate = torch.exp(s["a_log"].double())
    z = _dt_of(s, case).double() + s["dt_bias"].double()
    delta = torch.logaddexp(z, torch.zeros_like(z))
    a = torch.exp(-rate * delta)
    skip = s["D"].double()[:, None]
    if op == "step":
        rows = torch.cat([s["tail"].double(), s["proj"][:, None, :C].double()], 1)
        pre = bias + torch.einsum("bwc,cw->bc", rows, w)
        x, b, c = _split(pre * torch.sigmoid(pre), case)
        b, c = (v[:, :, None].expand(-1, -1, H // G, -1).reshape(-1, H, M) for v in (b, c))
        X = a[..., None, None] * s["state"].double() + torch.einsum("bh,bhm,bhd->bhmd", delta, b, x)
        return {"y": torch.einsum("bhm,bhmd->bhd", c, X) + skip * x, "state": X, "tail": rows[:, 1:]}
    B, N = case["B"], case["N"]
    if op == "scan_bwd" and B * N * H * M * d * 8 > 40 << 30:
        return None
    x, b, c = (v.double() for v in _split(s["xbc"], case))
    b, c = (v[:, :, :, None].expand(-1, -1, -1, H // G, -1).reshape(B, N, H, M) for v in (b, c))
    X = torch.zeros(B, H, M, d, dtype=torch.float64, device=x.device)
    if s.get("state_in") is not None:
        X = s["state_in"].double()
    if op == "scan":
        y = torch.empty(B, N, H, d, dtype=torch.float64, device=x.device)
        for t in range(N):
            X = a[:, t, :, None, None] * X + (delta[:, t, :, None] * b[:, t])[..., None] * x[:, t, :, None]
            y[:, t] = (c[:, t, :, None] @ X)[:, :, 0]
        y += skip * x
        return {"y": y, "state": X} if case["state"] else {"y": y}
    dy = s["dy"].double()
    hist = torch.empty(N + 1, B, H, M, d, dtype=torch.float64, device=x.device)
    hist[0] = X
    for t in range(N):
        X = a[:, t, :, None, None] * X + (delta[:, t, :, None] * b[:, t])[..., None] * x[:, t, :, None]
        hist[t + 1] = X
    dx, db, dc = skip * dy, torch.empty_like(b), torch.empty_like(c)
    ddelta, drate = torch.empty_like(delta), torch.empty_like(delta)
    Z = torch.zeros_like(X)
    for t in range(N - 1, -1, -1):
        Z = Z + c[:, t, :, :, None] * dy[:, t, :, None]
        dc[:, t] = (hist[t + 1] @ dy[:, t, :, :, None])[..., 0]
        Zx = (Z @ x[:, t, :, :, None])[..., 0]
        db[:, t] = delta[:, t, :, None] * Zx
        dx[:, t] += delta[:, t, :, None] * (b[:, t, :, None] @ Z)[:, :, 0]
        Z = a[:, t, :, None, None] * Z
        lost = (Z * hist[t]).sum((-1, -2))  # d / d log a_t
        drate[:, t] = -delta[:, t] * lost
        ddelta[:, t] = (b[:, t] * Zx).sum(-1) - rate * lost
    dz = ddelta * torch.sigmoid(z)
    return {"dx": dx, "db": db.reshape(B, N, G, H // G, M).sum(3), "dc": dc.reshape(B, N, G, H // G, M).sum(3),
            "ddt": dz, "da_log": rate * drate.sum((0, 1)), "ddt_bias": dz.sum((0, 1)),
            "dD": (x * dy).sum((0, 1, 3))}
