"""The decoder's gated feed-forward block and its projections in 8 bits, as measured operators.

``listed()`` gives the measured cases and ``draw()`` more of the same ranges; ``prepare()`` makes a
case's inputs from a seed; ``run()`` makes one pass, either through the library (``own``) or in a
plain form of elementary torch operations; ``exact()`` evaluates the definition in 64 bits.

Operators (T rows of D channels, F hidden channels; weights [out, in] as a linear layer has them):

  ffn       g = x Wg^T, u = x Wu^T, h = g / (1 + e^-g) * u, out = h Wd^T; g, u and h kept for training
  ffn_bwd   dh = dy Wd, du = dh silu(g), dg = dh u silu'(g), dx = dg Wg + du Wu, dWg = dg^T x,
            dWu = du^T x, dWd = dy^T h, given x, dy and what the forward pass kept
  quant     q = x / scale in e4m3, scale = max |x| / 448 over 128 channels of one row, or of 128 rows
            (1 for zeros)
  gemm      out = (a sa) (b sb)^T, a [T, K] and b [N, K] in e4m3, a scale for 128 channels of each row
            of a and for each block of 128 x 128 of b
  glu       g and u of a and two such weights, h = silu(g) u quantised as by quant, a scale for 128
            channels of each row
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0


# ---- cases -------------------------------------------------------------------------------

def listed():
    return [
        # the 1.3B-like prompt at the training context (4 x 4096 positions, 16 heads of 128)
        dict(name="ffn_1p3b", op="ffn", dtype="bf16", T=16384, D=2048, F=5632, keep=False),
        # training the 125M-like layer (8 x 2048 positions, 12 heads of 64): what gradients need is kept
        dict(name="ffn_125m_train", op="ffn", dtype="bf16", T=16384, D=768, F=2048, keep=True),
        # one token of one sequence, where the weights' bytes and latency count
        dict(name="ffn_one", op="ffn", dtype="bf16", T=1, D=2048, F=5632, keep=False),
        # a short ragged fp32 prompt of two heads of 32
        dict(name="ffn_tiny_f32", op="ffn", dtype="f32", T=251, D=64, F=176, keep=True),
        # the 125M-like layer's gradients
        dict(name="ffn_bwd_125m", op="ffn_bwd", dtype="bf16", T=16384, D=768, F=2048),
        # a small fp32 training step with an odd number of rows
        dict(name="ffn_bwd_f32", op="ffn_bwd", dtype="f32", T=509, D=128, F=344),
        # a tensor of weights laid out for 8 bits, when they are loaded or were updated
        dict(name="quant_weights", op="quant", dtype="bf16", T=5632, D=2048, rows=128),
        # activations of an odd number of positions ahead of a projection
        dict(name="quant_rows", op="quant", dtype="bf16", T=4099, D=5632, rows=1),
        # the selective mixer's projection to [x | b | c | dt] of the 1.3B-like prompt: 2048 + 128 + 16 channels
        dict(name="gemm_1p3b", op="gemm", out="bf16", T=16384, K=2048, N=2192),
        # the projection back to the stream, for a few decoded tokens
        dict(name="gemm_decode", op="gemm", out="bf16", T=5, K=5632, N=2048),
        # the feed-forward block's first half in 8 bits: a long prompt continued to 14336 positions
        dict(name="glu_14k", op="glu", T=14336, D=2048, F=5632),
        # the same for the decode batch of 256 sequences
        dict(name="glu_256", op="glu", T=256, D=2048, F=5632),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_bwd", "quant", "gemm", "gemm", "glu"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    if op == "quant":
        T, D = _log(rng, 1, 16384), 16 * _log(rng, 2, 512)
        return dict(op=op, dtype=dtype, T=min(T, 4099 * 5632 // D), D=D, rows=rng.choice([1, 128]))
    if op == "gemm":
        K, N = 16 * _log(rng, 4, 352), 8 * _log(rng, 4, 704)
        return dict(op=op, out="f32" if rng.random() < 0.2 else "bf16", T=_log(rng, 1, min(16384, 16384 * 2048 * 2192 // (K * N))),
                    K=K, N=N)
    if op == "glu":
        D, F = 16 * _log(rng, 4, 128), 16 * _log(rng, 4, 352)
        return dict(op=op, T=_log(rng, 1, min(14336, 14336 * 2048 * 5632 // (D * F))), D=D, F=F)
    D, F = 8 * _log(rng, 4, 256), 8 * _log(rng, 8, 704)
    most = 16384 * (2048 * 5632 if op == "ffn" else 768 * 2048) // (D * F)
    T = _log(rng, 1, max(1, min(16384, most // (8 if dtype == "f32" else 1))))
    case = dict(op=op, dtype=dtype, T=T, D=D, F=F)
    return {**case, "keep": rng.random() < 0.5} if op == "ffn" else case


# ---- inputs ------------------------------------------------------------------------------

def _blocks(n):
    return (n + 127) // 128


def _quantised(x, rows):
    """q in e4m3 and its scales, one for 128 channels of `rows` rows."""
    T, K = x.shape
    n, k = (T + rows - 1) // rows, _blocks(K)
    full = x.float().new_zeros(n * rows, k * 128)
    full[:T, :K] = x
    v = full.unflatten(0, (n, rows)).unflatten(2, (k, 128))
    top = v.abs().amax((1, 3))
    scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    q = torch.clamp(v / scale[:, None, :, None], -E4M3_MAX, E4M3_MAX).flatten(2).flatten(0, 1)[:T, :K]
    return q.to(E4M3).contiguous(), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)

    def randn(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    op = case["op"]
    s = {"case": case}
    if op == "quant":
        # channels of unlike size, as activations and weights have them
        s["x"] = (randn(case["T"], case["D"]) * torch.exp(randn(case["D"]))).to(_DT[case["dtype"]])
        return s
    if op == "gemm":
        s["a"], s["sa"] = _quantised(randn(case["T"], case["K"]), 1)
        s["b"], s["sb"] = _quantised(randn(case["N"], case["K"], scale=case["K"] ** -0.5), 128)
        return s
    T, D, F = case["T"], case["D"], case["F"]
    if op == "glu":
        s["a"], s["sa"] = _quantised(randn(T, D), 1)
        s["wg"], s["sg"] = _quantised(randn(F, D, scale=D ** -0.5), 128)
        s["wu"], s["su"] = _quantised(randn(F, D, scale=D ** -0.5), 128)
        return s
    dt = _DT[case["dtype"]]
    s["x"] = randn(T, D).to(dt)
    s["wg"], s["wu"] = randn(F, D, scale=D ** -0.5).to(dt), randn(F, D, scale=D ** -0.5).to(dt)
    s["wd"] = randn(D, F, scale=F ** -0.5).to(dt)
    if op == "ffn_bwd":
        s["dy"] = randn(T, D).to(dt)
        gate, up = s["x"].float() @ s["wg"].float().t(), s["x"].float() @ s["wu"].float().t()
        s["acts"] = torch.stack([gate, up, _silu(gate) * up]).to(dt)
    return s


# ---- the library -------------------------------------------------------------------------

def _run_own(s):
    from linear_token_mixer_sc_gb300 import binding

    case = s["case"]
    op = case["op"]
    if op == "ffn":
        out, acts = binding.ida_ffn(s["x"], s["wg"], s["wu"], s["wd"], acts=case["keep"])
        return {"out": out, "acts": acts} if case["keep"] else {"out": out}
    if op == "ffn_bwd":
        g = binding.ida_ffn_backward(s["x"], s["wg"], s["wu"], s["wd"], s["acts"], s["dy"])
        return {"dx": g["x"], "dwg": g["w_gate"], "dwu": g["w_up"], "dwd": g["w_down"]}
    if op == "quant":
        q, scale = binding.ida_quant_e4m3(s["x"], rows=case["rows"])
        return {"q": q, "scale": scale}
    if op == "gemm":
        return {"out": binding.ida_gemm_e4m3(s["a"], s["sa"], s["b"], s["sb"], dtype=_DT[case["out"]])}
    q, scale = binding.ida_glu_e4m3(s["a"], s["sa"], s["wg"], s["sg"], s["wu"], s["su"])
    return {"q": q, "scale": scale}


# ---- the plain forms ---------------------------------------------------------------------

def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _values(q, scale, rows):
    """The values that q and its scales stand for, in 32 bits."""
    T, K = q.shape
    return q.float() * scale.repeat_interleave(rows, 0)[:T].repeat_interleave(128, 1)[:, :K]


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quant":
        q, scale = _quantised(s["x"], case["rows"])
        return {"q": q, "scale": scale}
    if op == "gemm":
        return {"out": (_values(s["a"], s["sa"], 1) @ _values(s["b"], s["sb"], 128).t()).to(_DT[case["out"]])}
    if op == "glu":
        a = _values(s["a"], s["sa"], 1)
        h = _silu(a @ _values(s["wg"], s["sg"], 128).t()) * (a @ _values(s["wu"], s["su"], 128).t())
        q, scale = _quantised(h, 1)
        return {"q": q, "scale": scale}
    dt = _DT[case["dtype"]]
    x, wg, wu, wd = (s[k].float() for k in ("x", "wg", "wu", "wd"))
    if op == "ffn":
        gate, up = x @ wg.t(), x @ wu.t()
        h = _silu(gate) * up
        out = (h @ wd.t()).to(dt)
        return {"out": out, "acts": torch.stack([gate, up, h]).to(dt)} if case["keep"] else {"out": out}
    dy = s["dy"].float()
    gate, up, h = (t.float() for t in s["acts"])
    sig = 1.0 / (1.0 + torch.exp(-gate))
    dh = dy @ wd
    du = dh * gate * sig
    dg = dh * up * sig * (1.0 + gate * (1.0 - sig))
    return {"dx": (dg @ wg + du @ wu).to(dt), "dwg": (dg.t() @ x).to(dt), "dwu": (du.t() @ x).to(dt),
            "dwd": (dy.t() @ h).to(dt)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "gemm":
        T, K, N = case["T"], case["K"], case["N"]
        return {"bytes": T * K + N * K + 4 * _blocks(K) * (T + _blocks(N)) + T * N * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * T * K * N}
    T, D = case["T"], case["D"]
    if op == "quant":
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": T * D * (e + 1) + 4 * _blocks(D) * -(-T // case["rows"]), "flops": 2 * T * D}
    F = case["F"]
    if op == "glu":
        return {"bytes": T * D + 2 * D * F + T * F + 4 * (T * (_blocks(D) + _blocks(F)) + 2 * _blocks(D) * _blocks(F)),
                "flops": 4 * T * D * F + 6 * T * F}
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "ffn":
        return {"bytes": e * (2 * T * D + 3 * D * F + (3 * T * F if case["keep"] else 0)), "flops": 6 * T * D * F + 4 * T * F}
    return {"bytes": e * (3 * T * D + 3 * T * F + 6 * D * F), "flops": 12 * T * D * F + 12 * T * F}


# ---- the definitions in 64 bits ------------------------------------------------------------

def _exact_values(q, scale, rows):
    r = torch.arange(q.shape[0], device=q.device) // rows
    c = torch.arange(q.shape[1], device=q.device) // 128
    return q.double() * scale.double()[r][:, c]


def _exact_quant(x, rows):
    """Scales, and the quotients that e4m3 rounds."""
    x = x.double()
    T, K = x.shape
    n, k = -(-T // rows), _blocks(K)
    r, c = torch.arange(T, device=x.device) // rows, torch.arange(K, device=x.device) // 128
    top = torch.zeros(n * k, dtype=x.dtype, device=x.device)
    top = top.scatter_reduce(0, (r[:, None] * k + c).reshape(-1), x.abs().reshape(-1), "amax").reshape(n, k)
    scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    return {"q": x / scale[r][:, c], "scale": scale}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        return _exact_quant(s["x"], case["rows"])
    if op == "gemm":
        return {"out": torch.einsum("tk,nk->tn", _exact_values(s["a"], s["sa"], 1), _exact_values(s["b"], s["sb"], 128))}
    if op == "glu":
        a = _exact_values(s["a"], s["sa"], 1)
        gate = torch.einsum("td,fd->tf", a, _exact_values(s["wg"], s["sg"], 128))
        return _exact_quant(gate * torch.sigmoid(gate) * torch.einsum("td,fd->tf", a, _exact_values(s["wu"], s["su"], 128)), 1)
    x, wg, wu, wd = (s[k].double() for k in ("x", "wg", "wu", "wd"))
    if op == "ffn":
        gate, up = torch.einsum("td,fd->tf", x, wg), torch.einsum("td,fd->tf", x, wu)
        h = gate * torch.sigmoid(gate) * up
        out = torch.einsum("tf,df->td", h, wd)
        return {"out": out, "acts": torch.stack([gate, up, h])} if case["keep"] else {"out": out}
    dy = s["dy"].double()
    gate, up, h = s["acts"].double().unbind()
    sig = torch.sigmoid(gate)
    dh = torch.einsum("td,df->tf", dy, wd)
    dg, du = dh * up * (sig + gate * sig * (1 - sig)), dh * gate * sig
    return {"dx": torch.einsum("tf,fd->td", dg, wg) + torch.einsum("tf,fd->td", du, wu),
            "dwg": torch.einsum("tf,td->fd", dg, x), "dwu": torch.einsum("tf,td->fd", du, x),
            "dwd": torch.einsum("td,tf->df", dy, h)}
