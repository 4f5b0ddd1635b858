"""The selective mixer at finite inputs far from the usual ones: positions that forget everything, long
runs of them, arguments where a sigmoid is small.

Bounds as in ``test_gpu_ssm.py`` where nothing else is said.
"""
import math

import pytest
import torch

from linear_token_mixer_sc_gb300 import binding, build
from tests import ssm_cases as sc
from tests.ssm_cases import DT, U32, worst
from tests.test_gpu_ssm import _done, _on_gpu, _scan_bounds, _scan_inputs, _scan_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


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
