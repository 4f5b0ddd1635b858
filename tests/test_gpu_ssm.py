"""GPU parity of the selective mixer (ida_ssm_conv, ida_ssm_scan, ida_ssm_step and the backward
calls) against the fp64 oracle ``oracle/ida_ssm.py``, element by element.

Every bound is a count of roundings: half a step of the output's type on the value, plus, times
the sum of the absolute terms behind the value (the oracle on absolute inputs):
- fp32 arithmetic: 2^-24 per operation, at most 8 N + 64 of them along a sequence of N positions
  (products, sums, the decay and step size of each position);
- bf16 tensor-core operands: 2^-8 for each operand rounded to bf16 (at most two meet in a term
  of y, three in one of a gradient), 2^-16 for one kept as the sum of two bf16 values (states
  and what the fp32 gradients of parameters are summed from; two such operands may meet there).
"""
import pytest
import torch

from linear_token_mixer_sc_gb300 import binding, build
from oracle import ida_ssm as orc
from tests import ssm_cases as sc
from tests.ssm_cases import HALF, U32, worst

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


def _done():
    torch.cuda.synchronize()
    assert binding.ida_device_error() == 0


# ---- the convolution ---------------------------------------------------------------------------

# (B, N, C, W, dtype, state): one position, fewer positions than taps, strip and batch edges
CONVS = [(1, 1, 8, 4, "bf16", True), (2, 2, 24, 4, "f32", True), (3, 3, 40, 4, "bf16", False),
         (2, 7, 64, 3, "f32", False), (1, 33, 136, 2, "bf16", True), (2, 65, 72, 4, "f32", True),
         (1, 257, 1024, 4, "bf16", True), (2, 31, 16, 1, "bf16", False), (70, 9, 512, 4, "bf16", False)]


def _conv_inputs(B, N, C, W, dtype, state, seed=3):
    p = sc.params(1, C, W, seed)
    row = sc.rows(B, N, C, 5, dtype, seed + 1)
    s = torch.randn(B, W - 1, C, generator=sc.gen(seed + 2)) if state else None
    return p, row, s


def _conv_error(pre_abs, out, dtype, W):
    # SiLU's slope is below 1.1; the hardware exponential and reciprocal are within 2^-20
    return HALF[dtype] * out.abs() + 1.1 * (W + 2) * U32 * pre_abs + (2.0 ** -20 if dtype == "bf16" else 8 * U32) * out.abs()


@pytest.mark.parametrize("case", CONVS, ids=str)
def test_conv(case):
    B, N, C, W, dtype, state = case
    p, row, s = _conv_inputs(*case)
    out, tail = binding.ida_ssm_conv(row.cuda()[..., :C], p["conv_w"].cuda(), p["conv_b"].cuda(),
                                     state_in=None if s is None else s.cuda(), final_state=True)
    _done()
    x, w, b = row[..., :C].double(), p["conv_w"].double(), p["conv_b"].double()
    ref, rtail = orc.conv(x, w, b, None if s is None else s.double())
    head = torch.zeros(B, W - 1, C, dtype=torch.float64) if s is None else s.double()
    rows = torch.cat([head, x], 1)
    pre_abs = b.abs() + sum(w[:, j].abs() * rows[:, j:j + N].abs() for j in range(W))
    assert worst(out, ref, _conv_error(pre_abs, ref, dtype, W)) <= 1
    assert torch.equal(tail.cpu().double(), rtail)


@pytest.mark.parametrize("case", [c for c in CONVS if not c[5]] + [(1, 130, 48, 4, "f32", False),
                                                                  (2, 64, 260 * 8, 4, "bf16", False),
                                                                  (1, 1, 8, 4, "bf16", False)], ids=str)
def test_conv_backward(case):
    B, N, C, W, dtype, _ = case
    p, row, _ = _conv_inputs(*case)
    dout = torch.randn(B, N, C, generator=sc.gen(8)).to(sc.DT[dtype])
    wide = torch.zeros(B, N, C + 16, dtype=sc.DT[dtype], device="cuda")
    g = binding.ida_ssm_conv_backward(row.cuda()[..., :C], dout.cuda(), p["conv_w"].cuda(), p["conv_b"].cuda(),
                                      dx=wide[..., :C])
    _done()
    x, w, b = row[..., :C].double(), p["conv_w"].double(), p["conv_b"].double()
    rx, rw, rb = orc.grads(lambda *v: orc.conv(*v)[0], [x, w, b], dout.double())
    # |SiLU'| <= 1.1, |SiLU''| <= 0.5: the error of one position's gradient at the convolution
    head = torch.zeros(B, W - 1, C, dtype=torch.float64)
    rows = torch.cat([head, x], 1)
    pre_abs = b.abs() + sum(w[:, j].abs() * rows[:, j:j + N].abs() for j in range(W))
    eg = dout.double().abs() * U32 * (0.5 * (W + 2) * pre_abs + 16 * (1 + pre_abs))
    ga = 1.1 * dout.double().abs()

    def back(v, wt):  # sum over the taps of position t + W-1-j
        o = torch.zeros_like(v)
        for j in range(W):
            k = W - 1 - j
            if k < N:
                o[:, :N - k] += wt[:, j] * v[:, k:]
        return o

    assert worst(g["x"], rx, HALF[dtype] * rx.abs() + back(eg, w.abs()) + W * U32 * back(ga, w.abs())) <= 1
    n = 64 + 8 + (B * N + 511) // 512 + 8  # additions behind one sum: a strip, its block, the blocks
    ew = torch.stack([((eg + n * U32 * ga) * rows[:, j:j + N].abs()).sum((0, 1)) for j in range(W)], -1)
    assert worst(g["conv_w"], rw, ew + U32 * rw.abs()) <= 1
    assert worst(g["conv_b"], rb, (eg + n * U32 * ga).sum((0, 1)) + U32 * rb.abs()) <= 1
    assert not wide[..., C:].any()


# ---- the scan ----------------------------------------------------------------------------------

# (B, N, H, d, G, M, dtype, state, fast)
SCANS = [
    (1, 1, 1, 8, 1, 8, "bf16", True, False),        # one position, the smallest head
    (2, 15, 2, 32, 1, 16, "f32", False, False),      # inside one tile
    (1, 64, 2, 64, 2, 64, "bf16", True, False),      # whole tiles
    (1, 128, 1, 128, 1, 64, "bf16", True, False),
    (2, 129, 3, 64, 1, 128, "bf16", False, False),   # one position behind a tile, heads shared
    (1, 200, 4, 128, 2, 64, "bf16", True, False),
    (1, 131, 2, 256, 1, 24, "bf16", True, False),    # the widest head, a row of states that is no power of two
    (1, 70, 2, 200, 2, 104, "f32", True, False),
    (1, 97, 5, 72, 5, 40, "bf16", False, False),
    (1, 300, 2, 40, 1, 128, "f32", False, False),    # the most states; split across SMs
    (2, 530, 1, 64, 1, 64, "bf16", True, False),     # several segments
    (1, 777, 2, 128, 1, 128, "bf16", True, False),
    (1, 260, 2, 64, 1, 64, "bf16", True, True),      # decays that underflow within a tile
    (1, 150, 2, 32, 1, 32, "f32", True, True),
]


def _scan_inputs(B, N, H, d, G, M, dtype, state, fast, seed=5):
    C = H * d + 2 * G * M
    p = sc.params(H, 8, 1, seed, fast)
    row = sc.rows(B, N, C, H, dtype, seed + 1)
    s = torch.randn(B, H, M, d, generator=sc.gen(seed + 2)) * 0.3 if state else None
    return p, row, s, C


def _on_gpu(row, C, H, d, G, M):
    r = row.cuda()
    return (*sc.split(r[..., :C], H, d, G, M), r[..., C:C + H])


def _scan_ref(row, C, H, d, G, M, p, s, absolute=False):
    x, b, c = sc.split(row[..., :C].double(), H, d, G, M)
    D, q = p["D"].double(), sc.to64(p)
    if absolute:
        x, b, c, D, s = x.abs(), b.abs(), c.abs(), D.abs(), None if s is None else s.abs()
    return orc.scan(x, b, c, row[..., C:C + H].double(), q["a_log"], q["dt_bias"], D,
                    None if s is None else s.double())


def _scan_bounds(dtype, N, y, ya, Xa):
    chain = (8 * N + 64) * U32
    op = 2.05 * 2.0 ** -8 if dtype == "bf16" else 0.0
    return HALF[dtype] * y.abs() + (op + chain) * ya, ((2.0 ** -16 if dtype == "bf16" else 0.0) + chain) * Xa


@pytest.mark.parametrize("split", [True, False], ids=["workspace", "no workspace"])
@pytest.mark.parametrize("case", SCANS, ids=str)
def test_scan(case, split):
    B, N, H, d, G, M, dtype, state, fast = case
    p, row, s, C = _scan_inputs(*case)
    ws = None if split else torch.empty(0, dtype=torch.uint8, device="cuda")
    y, X = binding.ida_ssm_scan(*_on_gpu(row, C, H, d, G, M), sc.cuda(p), state_in=None if s is None else s.cuda(),
                                final_state=True, workspace=ws)
    _done()
    ry, rX = _scan_ref(row, C, H, d, G, M, p, s)
    ya, Xa = _scan_ref(row, C, H, d, G, M, p, s, absolute=True)
    by, bX = _scan_bounds(dtype, N, ry, ya, Xa)
    assert worst(y, ry, by) <= 1
    assert worst(X, rX, bX) <= 1


def test_scan_without_final_state_gives_the_same_outputs():
    case = SCANS[5]
    p, row, s, C = _scan_inputs(*case)
    args = (*_on_gpu(row, C, *case[2:6]), sc.cuda(p))
    y, X = binding.ida_ssm_scan(*args, state_in=s.cuda(), final_state=True)
    z, none = binding.ida_ssm_scan(*args, state_in=s.cuda())
    _done()
    assert none is None and torch.equal(y, z)


def test_scan_of_no_positions_hands_the_state_on():
    s = torch.randn(2, 3, 16, 8, device="cuda")
    e = torch.empty(2, 0, 3, 8, device="cuda")
    bc = torch.empty(2, 0, 1, 16, device="cuda")
    p = sc.cuda(sc.params(3, 8, 1, 1))
    y, X = binding.ida_ssm_scan(e, bc, bc, e[..., 0], p, state_in=s, final_state=True)
    _, Z = binding.ida_ssm_scan(e, bc, bc, e[..., 0], p, final_state=True)
    _done()
    assert y.numel() == 0 and torch.equal(X, s) and not Z.any()
    x = torch.empty(2, 0, 16, device="cuda")
    t = torch.randn(2, 3, 16, device="cuda")
    w = torch.randn(16, 4, device="cuda")
    _, T = binding.ida_ssm_conv(x, w, w[:, 0].contiguous(), state_in=t, final_state=True)
    _done()
    assert torch.equal(T, t)


def test_scan_leaves_other_heads_alone_when_one_is_not_finite():
    """A NaN in one head's x, dt or state reaches that head's outputs only."""
    case = (1, 140, 3, 64, 1, 64, "bf16", True, False)
    B, N, H, d, G, M = case[:6]
    p, row, s, C = _scan_inputs(*case)
    y0, X0 = binding.ida_ssm_scan(*_on_gpu(row, C, H, d, G, M), sc.cuda(p), state_in=s.cuda(), final_state=True)
    bad = row.clone()
    bad[0, 70, d + 3] = float("nan")      # x of head 1
    bad[0, 20, C + 1] = float("inf")      # dt of head 1
    s1 = s.clone()
    s1[0, 1, 2, 5] = float("inf")
    y1, X1 = binding.ida_ssm_scan(*_on_gpu(bad, C, H, d, G, M), sc.cuda(p), state_in=s1.cuda(), final_state=True)
    _done()
    for h in (0, 2):
        assert torch.equal(y0[:, :, h], y1[:, :, h]) and torch.equal(X0[:, h], X1[:, h])


# ---- one position ------------------------------------------------------------------------------

# (B, H, d, G, M, W, dtype)
STEPS = [(1, 1, 8, 1, 8, 4, "bf16"), (3, 16, 128, 1, 64, 4, "bf16"), (2, 6, 72, 3, 128, 3, "f32"),
         (1, 24, 64, 2, 64, 2, "bf16"), (2, 3, 256, 1, 40, 1, "f32"), (5, 5, 128, 5, 128, 4, "f32"),
         (1, 33, 16, 1, 16, 4, "bf16")]


@pytest.mark.parametrize("case", STEPS, ids=str)
def test_steps(case):
    """Five positions in a row, the states carried on the GPU, against the oracle's five."""
    B, H, d, G, M, W, dtype = case
    C = H * d + 2 * G * M
    p = sc.params(H, C, W, 7)
    tail = torch.randn(B, W - 1, C, generator=sc.gen(1))
    X = torch.randn(B, H, M, d, generator=sc.gen(2)) * 0.3
    dp, dtail, dX = sc.cuda(p), tail.cuda(), X.cuda()
    p64, t64, X64, Xa = sc.to64(p), tail.double(), X.double(), X.double().abs()
    pa = {k: (v.abs() if k == "D" else v) for k, v in p64.items()}
    for k in range(5):
        row = sc.rows(B, 1, C, H, dtype, 40 + k)[:, 0]
        r = row.cuda()
        y = binding.ida_ssm_step(r[:, :C], r[:, C:C + H], dp, dtail, dX, G)
        _done()
        x64, dt64 = row[:, :C].double(), row[:, C:C + H].double()
        act = orc.conv(x64[:, None], p64["conv_w"], p64["conv_b"], t64)[0]
        xa, ba, ca = sc.split(act.abs(), H, d, G, M)
        ya, Xa = orc.scan(xa, ba, ca, dt64[:, None], pa["a_log"], pa["dt_bias"], pa["D"], Xa)
        ry, t64, X64 = orc.step(x64, dt64, p64, t64, X64, G)
        # the convolved values are within (W + 10) 2^-24 of sums up to a few times their size: 64
        # roundings for each of two factors; M products are summed; k positions have gone before
        n = (2 * 64 * 8 + M + 16 * (k + 1)) * U32
        # a convolved value near zero has lost its relative accuracy: absolute terms of its window
        big = act.abs().amax() * 64 * U32 * (1 + X64.abs().amax() + act.abs().amax())
        assert worst(y, ry, HALF[dtype] * ry.abs() + n * ya[:, 0] + big * M) <= 1
        assert worst(dX, X64, n * Xa + big) <= 1
        assert torch.equal(dtail.cpu().double(), t64)


# ---- the scan's gradients ------------------------------------------------------------------------

# (B, N, H, d, G, M, dtype, state, fast)
GRADS = [
    (1, 1, 1, 8, 1, 8, "bf16", False, False), (2, 9, 2, 32, 1, 16, "f32", False, False),
    (1, 64, 2, 64, 2, 64, "bf16", False, False), (1, 65, 2, 64, 1, 64, "bf16", False, False),
    (2, 130, 3, 128, 1, 64, "bf16", False, False), (1, 70, 2, 256, 1, 128, "f32", False, False),
    (1, 128, 2, 128, 1, 128, "bf16", False, False), (1, 77, 4, 40, 2, 24, "f32", False, False),
    (2, 190, 2, 72, 1, 40, "bf16", False, False), (1, 100, 2, 64, 1, 64, "bf16", False, True),
    (1, 90, 2, 32, 2, 32, "f32", False, True), (1, 140, 1, 256, 1, 128, "bf16", False, False),
    (2, 150, 4, 64, 2, 128, "bf16", False, False), (1, 200, 6, 128, 1, 104, "bf16", False, False),
    (1, 260, 3, 16, 3, 72, "bf16", False, True), (1, 300, 5, 64, 1, 16, "bf16", False, False),
    (1, 20, 70, 8, 1, 16, "bf16", False, False),  # one CTA's heads are more than two batches of rates
]
NAMES = ("x", "b", "c", "dt", "a_log", "dt_bias", "D")


@pytest.mark.parametrize("case", GRADS, ids=str)
def test_scan_backward(case):
    B, N, H, d, G, M, dtype, _, fast = case
    p, row, _, C = _scan_inputs(*case)
    dy = torch.randn(B, N, H, d, generator=sc.gen(11)).to(sc.DT[dtype])
    g = binding.ida_ssm_scan_backward(*_on_gpu(row, C, H, d, G, M), sc.cuda(p), dy.cuda())
    _done()
    x, b, c = (t.contiguous() for t in sc.split(row[..., :C].double(), H, d, G, M))
    q = sc.to64(p)
    leaves = [x, b, c, row[..., C:C + H].double(), q["a_log"], q["dt_bias"], q["D"]]
    ref = orc.grads(lambda *v: orc.scan(*v)[0], leaves, dy.double())
    size = orc.scan_grad_sizes(*leaves, dy.double())
    chain = (8 * N + 2 * d + 2 * M + 64) * U32
    for k, name in enumerate(NAMES):
        if k < 4:  # stored in dtype; bf16 operands on the tensor cores
            bound = HALF[dtype] * ref[k].abs() + ((3.1 * 2.0 ** -8 if dtype == "bf16" else 0.0) + chain) * size[k]
        else:
            bound = ((2.0 ** -15 if dtype == "bf16" else 0.0) + chain) * size[k]
        assert worst(g[name], ref[k], bound) <= 1, name


def test_scan_backward_is_deterministic_and_agrees_with_differences():
    """The fp32 gradients against differences of the library's own forward pass."""
    case = (1, 40, 2, 16, 1, 16, "f32", False, False)
    B, N, H, d, G, M = case[:6]
    p, row, _, C = _scan_inputs(*case)
    args, dp = _on_gpu(row, C, H, d, G, M), sc.cuda(p)
    dy = torch.randn(B, N, H, d, generator=sc.gen(12)).cuda()
    g = binding.ida_ssm_scan_backward(*args, dp, dy)
    again = binding.ida_ssm_scan_backward(*args, dp, dy)
    for k in NAMES:
        assert torch.equal(g[k], again[k])

    def loss(dev_args, dev_p):
        return float((binding.ida_ssm_scan(*dev_args, dev_p)[0].double() * dy.double()).sum())

    size = float(sum(t.abs().sum() for t in (binding.ida_ssm_scan(*args, dp)[0] * dy,)))
    for k, t in (("x", args[0]), ("b", args[1]), ("c", args[2]), ("dt", args[3])):
        i = 0 if k != "dt" else 3
        way = torch.randn(t.shape, generator=sc.gen(20 + i)).cuda()
        e = 2.0 ** -7
        j = ("x", "b", "c", "dt").index(k)
        up = [v if n != j else (v + e * way) for n, v in enumerate(args)]
        dn = [v if n != j else (v - e * way) for n, v in enumerate(args)]
        diff = (loss(up, dp) - loss(dn, dp)) / (2 * e)
        # rounding of two losses over 2 e, and the third derivative along `way` times e^2 / 6,
        # both well below a hundredth of the terms' sum
        assert abs(diff - float((g[k].double() * way.double()).sum())) <= 1e-2 * size, k
    for k in ("a_log", "dt_bias", "D"):
        way = torch.randn(H, generator=sc.gen(30)).cuda()
        e = 2.0 ** -7
        diff = (loss(args, {**dp, k: dp[k] + e * way}) - loss(args, {**dp, k: dp[k] - e * way})) / (2 * e)
        assert abs(diff - float((g[k].double() * way.double()).sum())) <= 1e-2 * size, k


# ---- together, and how they are called -------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_block_over_a_prompt_and_its_next_positions(dtype):
    """Pre-norm of a residual stream, projection, convolution, scan and further single positions, as a
    decoder layer calls them, against the oracle of the same chain fed with each stage's own rounded
    input."""
    B, N, H, d, G, M, W, K = 2, 150, 4, 64, 2, 64, 4, 4
    C, D = H * d + 2 * G * M, 256
    R = (C + H + 7) // 8 * 8
    p = sc.params(H, C, W, 50)
    dp = sc.cuda(p)
    g = sc.gen(51)
    stream = torch.randn(B, N + K, D, generator=g).to(sc.DT[dtype]).cuda()
    add = torch.randn(B, N + K, D, generator=g).to(sc.DT[dtype]).cuda()
    w = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    proj_w = (torch.randn(D, R, generator=g) * D ** -0.5).to(sc.DT[dtype]).cuda()
    out, _, _, _ = binding.ida_rmsnorm(add, w, residual=stream)
    proj = out @ proj_w
    pre = proj[:, :N].contiguous()
    act, tail = binding.ida_ssm_conv(pre[..., :C], dp["conv_w"], dp["conv_b"], final_state=True)
    x, b, c = sc.split(act, H, d, G, M)
    y, X = binding.ida_ssm_scan(x, b, c, pre[..., C:C + H], dp, final_state=True)
    tail0, X0 = tail.clone(), X.clone()
    steps = [binding.ida_ssm_step(proj[:, N + k, :C], proj[:, N + k, C:C + H], dp, tail, X, G) for k in range(K)]
    _done()
    p64 = sc.to64(p)
    row = pre.cpu().double()
    ract, rtail = orc.conv(row[..., :C], p64["conv_w"], p64["conv_b"])
    assert torch.equal(tail0.cpu().double(), rtail)
    cut = torch.cat([act.cpu(), pre.cpu()[..., C:]], -1)  # the scan's own inputs
    ry, rX = _scan_ref(cut, C, H, d, G, M, p, None)
    ya, Xa = _scan_ref(cut, C, H, d, G, M, p, None, absolute=True)
    by, bX = _scan_bounds(dtype, N, ry, ya, Xa)
    assert worst(y, ry, by) <= 1 and worst(X0, rX, bX) <= 1
    # the steps from the library's own states, one more rounding chain behind them
    t64, X64 = tail0.cpu().double(), X0.cpu().double()
    tol = 2.0 ** -7 if dtype == "bf16" else 1e-5
    for k in range(K):
        r = proj[:, N + k].cpu().double()
        ry, t64, X64 = orc.step(r[:, :C], r[:, C:C + H], p64, t64, X64, G)
        assert float((steps[k].cpu().double() - ry).norm() / ry.norm()) <= tol
    assert float((X.cpu().double() - X64).norm() / X64.norm()) <= 1e-5


def test_gradients_of_conv_and_scan_together():
    """The scan's gradient rows go straight into the convolution's backward pass."""
    B, N, H, d, G, M, W = 1, 50, 2, 32, 1, 16, 4
    C = H * d + 2 * G * M
    p = sc.params(H, C, W, 60)
    dp = sc.cuda(p)
    row = sc.rows(B, N, C, H, "f32", 61)
    dev = row.cuda()
    act, _ = binding.ida_ssm_conv(dev[..., :C], dp["conv_w"], dp["conv_b"])
    dy = torch.randn(B, N, H, d, generator=sc.gen(62))
    gs = binding.ida_ssm_scan_backward(*sc.split(act, H, d, G, M), dev[..., C:C + H], dp, dy.cuda())
    gc = binding.ida_ssm_conv_backward(dev[..., :C], gs["xbc"], dp["conv_w"], dp["conv_b"])
    _done()
    p64 = sc.to64(p)

    def whole(x, w, b):
        return orc.scan(*sc.split(orc.conv(x, w, b)[0], H, d, G, M), row[..., C:C + H].double(), p64["a_log"],
                        p64["dt_bias"], p64["D"])[0]

    ref = orc.grads(whole, [row[..., :C].double(), p64["conv_w"], p64["conv_b"]], dy.double())
    for k, name in enumerate(("x", "conv_w", "conv_b")):
        # fp32 throughout: the relative error of a sum of a few hundred terms
        assert float((gc[name].cpu().double() - ref[k]).norm() / ref[k].norm()) <= 1e-5, name


def _all_calls(dtype):
    """name -> (tensors to be written, a call that writes them); outputs and workspaces made beforehand."""
    B, N, H, d, G, M, W = 2, 150, 4, 64, 2, 64, 4
    C = H * d + 2 * G * M
    p = sc.cuda(sc.params(H, C, W, 70))
    row = sc.rows(B, N, C, H, dtype, 71).cuda()
    x, b, c = sc.split(row[..., :C], H, d, G, M)
    dt = row[..., C:C + H]
    dy = torch.randn(B, N, H, d, generator=sc.gen(72)).to(sc.DT[dtype]).cuda()
    dout = torch.randn(B, N, C, generator=sc.gen(73)).to(sc.DT[dtype]).cuda()
    tail, X = torch.zeros(B, W - 1, C, device="cuda"), torch.zeros(B, H, M, d, device="cuda")

    def step():
        tail.zero_()
        X.zero_()
        y = binding.ida_ssm_step(row[:, 3, :C], dt[:, 3], p, tail, X, G)
        return [y, tail, X]

    def named(g):
        return [g[k] for k in sorted(g)]

    return {
        "conv": lambda: list(binding.ida_ssm_conv(row[..., :C], p["conv_w"], p["conv_b"], final_state=True)),
        "conv backward": lambda: named(binding.ida_ssm_conv_backward(row[..., :C], dout, p["conv_w"], p["conv_b"])),
        "scan": lambda: list(binding.ida_ssm_scan(x, b, c, dt, p, final_state=True)),
        "scan backward": lambda: named(binding.ida_ssm_scan_backward(x, b, c, dt, p, dy)),
        "step": step,
    }


@pytest.mark.parametrize("name", ["conv", "conv backward", "scan", "scan backward", "step"])
def test_captured_and_replayed(name):
    """A call captured into a CUDA graph and replayed gives what the eager call gives."""
    call = _all_calls("bf16")[name]
    ref = [t.clone() for t in call()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(2):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        _done()
        for a, b in zip(got, ref):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["conv", "conv backward", "scan", "scan backward", "step"])
def test_on_another_stream(name):
    call = _all_calls("bf16")[name]
    ref = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call()
    side.synchronize()
    for a, b in zip(got, ref):
        assert torch.equal(a, b)


def test_gradients_beside_the_inputs_in_the_same_rows():
    B, N, H, d, G, M = 2, 150, 4, 32, 2, 16
    C = H * d + 2 * G * M
    p = sc.cuda(sc.params(H, C, 4, 3))
    wide = torch.zeros(B, N, 2 * C, dtype=torch.bfloat16, device="cuda")
    wide[..., :C] = torch.randn(B, N, C, generator=sc.gen(5)).cuda()
    dout = torch.randn(B, N, C, generator=sc.gen(6)).bfloat16().cuda()
    want = binding.ida_ssm_conv_backward(wide[..., :C], dout, p["conv_w"], p["conv_b"])
    before = wide[..., :C].clone()
    got = binding.ida_ssm_conv_backward(wide[..., :C], dout, p["conv_w"], p["conv_b"], dx=wide[..., C:])
    assert torch.equal(got["x"], want["x"]) and torch.equal(wide[..., C:], want["x"])
    assert torch.equal(wide[..., :C], before) and torch.equal(got["conv_w"], want["conv_w"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_past_32_bits(dtype):
    """Slices of rows 2^26 elements apart, the last ones past element 2^32: the results of dense rows."""
    B, N, H, d, G, M, ld = 1, 70, 2, 32, 1, 16, 1 << 26
    C, row = H * d + 2 * G * M, (H * d + 2 * G * M + H + 7) // 8 * 8
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 20 GB")
    dense = sc.rows(B, N, C, H, dtype, 11).cuda()
    far = torch.empty(B * N * ld, dtype=dense.dtype, device="cuda").as_strided((B, N, row), (N * ld, ld, 1))
    far.copy_(dense)
    p = sc.cuda(sc.params(H, C, 4, 12))
    dout = torch.randn(B, N, C, generator=sc.gen(13)).to(dense.dtype).cuda()
    dy = torch.randn(B, N, H, d, generator=sc.gen(14)).to(dense.dtype).cuda()

    def run(rows):
        x, b, c = sc.split(rows[..., :C], H, d, G, M)
        dt = rows[..., C:C + H]
        out = list(binding.ida_ssm_conv(rows[..., :C], p["conv_w"], p["conv_b"], final_state=True))
        out += binding.ida_ssm_conv_backward(rows[..., :C], dout, p["conv_w"], p["conv_b"]).values()
        out += binding.ida_ssm_scan(x, b, c, dt, p, final_state=True)
        out += binding.ida_ssm_scan_backward(x, b, c, dt, p, dy).values()
        tail, state = torch.zeros(N, 3, C, device="cuda"), torch.zeros(N, H, M, d, device="cuda")
        return out + [binding.ida_ssm_step(rows[0, :, :C], dt[0], p, tail, state, G), tail, state]

    want, got = run(dense), run(far)
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    dx = far[..., :C]
    g = binding.ida_ssm_conv_backward(dense[..., :C], dout, p["conv_w"], p["conv_b"], dx=dx)
    assert torch.equal(g["x"], want[2]) and torch.equal(far[..., C:], dense[..., C:])


def test_outputs_stay_inside_their_rows():
    """Guard bands around y, the final state and the outputs of the step and the convolution."""
    B, N, H, d, G, M, W = 1, 131, 2, 72, 1, 40, 4
    C = H * d + 2 * G * M
    p = sc.cuda(sc.params(H, C, W, 80))
    row = sc.rows(B, N, C, H, "bf16", 81).cuda()
    x, b, c = sc.split(row[..., :C], H, d, G, M)
    raws = []

    def guarded(shape, dtype):
        n = 1
        for v in shape:
            n *= v
        raw = torch.full((n + 512,), 77.0, dtype=dtype, device="cuda")
        raws.append((raw, n))
        return raw[256:256 + n].view(shape)

    binding.ida_ssm_scan(x, b, c, row[..., C:C + H], p, final_state=guarded((B, H, M, d), torch.float32),
                         out=guarded((B, N, H, d), torch.bfloat16))
    binding.ida_ssm_conv(row[..., :C], p["conv_w"], p["conv_b"], final_state=guarded((B, W - 1, C), torch.float32),
                         out=guarded((B, N, C), torch.bfloat16))
    tail, X = guarded((B, W - 1, C), torch.float32), guarded((B, H, M, d), torch.float32)
    tail.zero_()
    X.zero_()
    binding.ida_ssm_step(row[:, 5, :C], row[:, 5, C:C + H], p, tail, X, G, out=guarded((B, H, d), torch.bfloat16))
    _done()
    for raw, n in raws:
        assert bool((raw[:256] == 77).all()) and bool((raw[256 + n:] == 77).all())
        assert bool(torch.isfinite(raw.float()).all())
