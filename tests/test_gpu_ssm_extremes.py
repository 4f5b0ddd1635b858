"""The selective mixer at finite inputs far from the usual ones: positions that forget everything, long
runs of them, rates at the end of fp32, arguments where a sigmoid is small; and its single position to
fp32 accuracy.

Bounds as in ``test_gpu_ssm.py`` where nothing else is said.
"""
import math

import pytest
import torch

from linear_token_mixer_sc_gb300 import binding, build
from oracle import ida_ssm as orc
from tests import ssm_cases as sc
from tests.ssm_cases import DT, HALF, U32, worst
from tests.test_gpu_ssm import NAMES, _done, _on_gpu, _scan_bounds, _scan_inputs, _scan_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


def check_scan_gradients(g, row, C, H, d, G, M, p, dy, dtype="bf16", sums=0):
    """`sums`: additions behind a parameter's gradient beside those along a sequence."""
    x, b, c = (t.contiguous() for t in sc.split(row[..., :C].double(), H, d, G, M))
    q = sc.to64(p)
    leaves = [x, b, c, row[..., C:C + H].double(), q["a_log"], q["dt_bias"], q["D"]]
    ref = orc.grads(lambda *v: orc.scan(*v)[0], leaves, dy.double())
    size = orc.scan_grad_sizes(*leaves, dy.double())
    chain = (8 * row.shape[1] + 2 * d + 2 * M + 64) * U32
    for k, name in enumerate(NAMES):
        if k < 4:
            bound = HALF[dtype] * ref[k].abs() + ((3.1 * 2.0 ** -8 if dtype == "bf16" else 0.0) + chain) * size[k]
        else:
            bound = ((2.0 ** -15 if dtype == "bf16" else 0.0) + chain + sums * U32) * size[k]
        assert worst(g[name], ref[k], bound) <= 1, name


def _large_steps(name, N, H):
    """(changes to the step sizes' inputs, changes to the parameters), by position and head."""
    at = torch.zeros(N, H)
    if name == "one step of 1e4 early":
        at[3] = 1e4
    elif name == "one step of 1e5 early":
        at[3] = 1e5
    elif name == "a step of 300 every 10 positions":
        at[::10] = 300.0
    elif name == "steps of 3e8 in one block of 16":
        at[16:32] = 3e8
    p = {}
    if name == "rates of e^7 and steps of 10":
        p = {"a_log": torch.full((H,), 7.0), "dt_bias": torch.full((H,), 10.0)}
    elif name == "rates of e^9 and steps of 10":
        p = {"a_log": torch.full((H,), 9.0), "dt_bias": torch.full((H,), 10.0)}
    else:
        p = {"a_log": torch.full((H,), math.log(16.0))}
    return at, p


LARGE = ["one step of 1e4 early", "one step of 1e5 early", "a step of 300 every 10 positions",
         "steps of 3e8 in one block of 16", "rates of e^7 and steps of 10", "rates of e^9 and steps of 10"]


def _large_case(name, dtype, N):
    case = (1, N, 2, 64, 1, 64, dtype, True, False)
    B, N, H, d, G, M = case[:6]
    p, row, s, C = _scan_inputs(*case)
    at, over = _large_steps(name, N, H)
    dt = row[0, :, C:C + H].float()
    row[0, :, C:C + H] = torch.where(at > 0, at, dt).to(DT[dtype])
    return row, s, C, {**p, **over}, (H, d, G, M)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", LARGE)
def test_scan_after_positions_that_forget(name, dtype):
    """A position's large decay takes nothing from the accuracy of the weights behind it."""
    row, s, C, p, shape = _large_case(name, dtype, 200)
    y, X = binding.ida_ssm_scan(*_on_gpu(row, C, *shape), sc.cuda(p), state_in=s.cuda(), final_state=True)
    _done()
    ry, rX = _scan_ref(row, C, *shape, p, s)
    ya, Xa = _scan_ref(row, C, *shape, p, s, absolute=True)
    by, bX = _scan_bounds(dtype, 200, ry, ya, Xa)
    assert worst(X, rX, bX) <= 1
    assert worst(y, ry, by) <= 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", LARGE)
def test_scan_gradients_after_positions_that_forget(name, dtype):
    row, _, C, p, shape = _large_case(name, dtype, 140)
    dy = torch.randn(1, 140, *shape[:2], generator=sc.gen(11)).to(DT[dtype])
    g = binding.ida_ssm_scan_backward(*_on_gpu(row, C, *shape), sc.cuda(p), dy.cuda())
    _done()
    check_scan_gradients(g, row, C, *shape, p, dy, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("split", [True, False], ids=["workspace", "no workspace"])
def test_state_behind_a_long_run_of_positions_that_forget(dtype, split):
    """More than 2048 positions of log2 a below -2^20 each: their sum passes 2^31."""
    B, N, H, d, G, M = 1, 4500, 1, 8, 1, 8
    p, row, s, C = _scan_inputs(B, N, H, d, G, M, dtype, True, False)
    p = {**p, "a_log": torch.full((H,), math.log(16.0))}
    row[..., C:C + H] = 2e5
    ws = None if split else torch.empty(0, dtype=torch.uint8, device="cuda")
    y, X = binding.ida_ssm_scan(*_on_gpu(row, C, H, d, G, M), sc.cuda(p), state_in=s.cuda(), final_state=True,
                                workspace=ws)
    _done()
    ry, rX = _scan_ref(row, C, H, d, G, M, p, s)
    ya, Xa = _scan_ref(row, C, H, d, G, M, p, s, absolute=True)
    by, bX = _scan_bounds(dtype, N, ry, ya, Xa)
    assert worst(X, rX, bX) <= 1
    assert worst(y, ry, by) <= 1


def test_fp32_conv_gradients_where_the_sigmoid_is_small():
    """One tap of 1 and no bias: the convolved value is the input, and each gradient one evaluation of
    SiLU' = s (1 + p (1 - s)).  e^-p within 2 units (4 u, u = 2^-24), the addition and the division
    make s good to 6 u; the product's terms then to (6 s + 1) u |p| s + 10 u |SiLU'|."""
    N, C = 600, 16
    x = (-30.0 * torch.rand(1, N, C, generator=sc.gen(1))).cuda()
    w, b = torch.ones(C, 1, device="cuda"), torch.zeros(C, device="cuda")
    g = binding.ida_ssm_conv_backward(x, torch.ones_like(x), w, b)
    _done()
    p = x.cpu().double()
    sg = torch.sigmoid(p)
    ref = sg * (1 + p * (1 - sg))
    bound = U32 * ((6 * sg + 1) * p.abs() * sg + 10 * ref.abs() + sg)
    assert worst(g["x"], ref, bound) <= 1


def _rates(name, H):
    """Parameters of heads whose decays are 0 at every step, or 1."""
    if name == "e^a_log above fp32":
        return {"a_log": torch.full((H,), 100.0)}
    if name == "e^a_log just within fp32":
        return {"a_log": torch.full((H,), 88.5)}
    return {"a_log": torch.full((H,), 60.0), "dt_bias": torch.full((H,), -60.0)}  # e^a_log times the step about 1


RATES = ["e^a_log above fp32", "e^a_log just within fp32", "a large rate and small steps"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", RATES)
def test_rates_at_the_end_of_the_range(name, dtype):
    """Finite a_log of any size: a prompt that ends inside a tile, its gradients, a position."""
    case = (1, 75, 2, 64, 1, 64, dtype, True, False)
    B, N, H, d, G, M = case[:6]
    p, row, s, C = _scan_inputs(*case)
    p = {**p, **_rates(name, H)}
    dp, args = sc.cuda(p), _on_gpu(row, C, H, d, G, M)
    y, X = binding.ida_ssm_scan(*args, dp, state_in=s.cuda(), final_state=True)
    dy = torch.randn(B, N, H, d, generator=sc.gen(11)).to(DT[dtype])
    g = binding.ida_ssm_scan_backward(*args, dp, dy.cuda())
    q = {**sc.params(H, C, 4, 9), **p, "conv_w": torch.zeros(C, 4), "conv_b": torch.randn(C, generator=sc.gen(9))}
    tail, Z = torch.zeros(N, 3, C, device="cuda"), s.cuda().expand(N, -1, -1, -1).contiguous()
    z = binding.ida_ssm_step(row[0, :, :C].cuda(), row[0, :, C:C + H].cuda(), sc.cuda(q), tail, Z, G)
    _done()
    ry, rX = _scan_ref(row, C, H, d, G, M, p, s)
    ya, Xa = _scan_ref(row, C, H, d, G, M, p, s, absolute=True)
    by, bX = _scan_bounds(dtype, N, ry, ya, Xa)
    assert worst(y, ry, by) <= 1
    assert worst(X, rX, bX) <= 1
    # the step's convolution is SiLU of the bias, a constant: one more rounding chain before the products
    rz, _, rZ = orc.step(row[0, :, :C].double(), row[0, :, C:C + H].double(), sc.to64(q),
                         torch.zeros(N, 3, C, dtype=torch.float64), s.double().expand(N, -1, -1, -1), G)
    ax, ab, ac = sc.split(orc.conv(torch.zeros(N, 1, C, dtype=torch.float64), sc.to64(q)["conv_w"], sc.to64(q)["conv_b"])[0].abs(),
                          H, d, G, M)
    za, Za = orc.scan(ax, ab, ac, row[0, :, None, C:C + H].double(), sc.to64(q)["a_log"], sc.to64(q)["dt_bias"],
                      sc.to64(q)["D"].abs(), s.double().abs().expand(N, -1, -1, -1))
    n = (M + 160) * U32
    # the step is off by (|z| + 10) u of itself, z its rounded argument, and the exponent of the decay E = rate
    # times step by 5 u more: the decay by a E (|z| + 15) u, which times the state before comes on top
    arg = row[0, :, C:C + H].double() + q["dt_bias"].double()
    E = torch.exp(q["a_log"].double()) * orc.step_size(row[0, :, C:C + H].double(), q["dt_bias"].double())
    far = (torch.exp(-E) * E * (arg.abs() + 15) * U32)[..., None, None] * s.double().abs()
    zfar = (ac[:, 0].repeat_interleave(H // G, 1)[..., None] * far).sum(2)
    assert worst(z, rz, HALF[dtype] * rz.abs() + n * za[:, 0] + zfar) <= 1
    assert worst(Z, rZ, n * Za + far) <= 1
    check_scan_gradients(g, row, C, H, d, G, M, p, dy, dtype)


# (B, H, d, G, M, W, dtype)
STEPS = [(2, 6, 72, 3, 128, 3, "f32"), (2, 3, 256, 1, 40, 1, "f32"), (3, 5, 128, 5, 64, 4, "f32"),
         (2, 12, 64, 1, 64, 4, "bf16"), (1, 24, 16, 2, 16, 2, "bf16")]


@pytest.mark.parametrize("case", STEPS, ids=str)
def test_steps_to_fp32_accuracy(case):
    """Three positions in a row, the error of every value followed through the formulas.  With u =
    2^-24: expf, log1pf within 2 units (4 u); pre by W + 1 multiply-adds; SiLU's slope is below 1.1
    and its evaluation is good to 7 u; softplus to u |z| + 10 u of its value."""
    B, H, d, G, M, W, dtype = case
    C, rep = H * d + 2 * G * M, H // G
    p = sc.params(H, C, W, 7)
    tail = torch.randn(B, W - 1, C, generator=sc.gen(1))
    X = torch.randn(B, H, M, d, generator=sc.gen(2)) * 0.3
    dp, dtail, dX = sc.cuda(p), tail.cuda(), X.cuda()
    q, t64, X64 = sc.to64(p), tail.double(), X.double()
    eX = torch.zeros_like(X64)
    rate = torch.exp(q["a_log"])
    for k in range(3):
        row = sc.rows(B, 1, C, H, dtype, 40 + k)[:, 0]
        r = row.cuda()
        y = binding.ida_ssm_step(r[:, :C], r[:, C:C + H], dp, dtail, dX, G)
        _done()
        x64, dt64 = row[:, :C].double(), row[:, C:C + H].double()
        rows = torch.cat([t64, x64[:, None]], 1)
        pre_abs = q["conv_b"].abs() + (q["conv_w"].abs().T * rows.abs()).sum(1)
        act = orc.conv(x64[:, None], q["conv_w"], q["conv_b"], t64)[0][:, 0]
        ea = 1.1 * (W + 1) * U32 * pre_abs + 7 * U32 * act.abs()
        (ax, ab, ac), (ex, eb, ec) = ([t.abs() for t in sc.split(v, H, d, G, M)] for v in (act, ea))
        ab, ac, eb, ec = (t.repeat_interleave(rep, 1)[..., None] for t in (ab, ac, eb, ec))
        ax, ex = ax[:, :, None], ex[:, :, None]
        delta = orc.step_size(dt64, q["dt_bias"])
        ed = U32 * ((dt64 + q["dt_bias"]).abs() + 10 * delta)
        decay = torch.exp(-rate * delta)
        edecay = decay * (5 * U32 * rate * delta + rate * ed + 4 * U32)
        delta, ed, decay, edecay = (t[..., None, None] for t in (delta, ed, decay, edecay))
        before = X64.abs()
        ry, t64, X64 = orc.step(x64, dt64, q, t64, X64, G)
        eX = (decay * eX + edecay * (before + eX) + delta * (ab * ex + eb * ax + eb * ex) +
              (ed + 3 * U32 * delta) * ab * ax + 2 * U32 * (X64.abs() + decay * before))
        D = q["D"].abs()[:, None]
        terms = (ac * X64.abs()).sum(2) + D * ax[:, :, 0]
        ey = ((ac + ec) * eX + ec * X64.abs()).sum(2) + D * ex[:, :, 0] + (M + 3) * U32 * terms
        assert worst(y, ry, HALF[dtype] * ry.abs() + ey) <= 1
        assert worst(dX, X64, eX + U32 * X64.abs()) <= 1
        assert torch.equal(dtail.cpu().double(), t64)
