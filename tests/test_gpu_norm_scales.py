"""The pre-norm's e4m3 output for groups of vanishing values."""
import pytest
import torch

from linear_token_mixer_sc_gb300 import binding, build
from oracle import ida_ssm as orc
from tests import ssm_cases as sc
from tests.ssm_cases import U32, worst

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 96])
@pytest.mark.parametrize("tiny", [1e-34, 1e-36, 1e-37, 1e-39, 1e-41, 1e-43, 1e-45])
def test_scales_of_vanishing_groups(tiny, group, dtype):
    """Groups of values around `tiny`, with exact zeros among them, beside ordinary groups.  A value
    below 2^-126 is stored to 2^-150; a scale is good to 2^-149 beside its relative error, and e4m3 to
    half a step: 2^-4 of the value, 2^-10 of the scale near zero."""
    rows, D = 5, 96
    x = torch.randn(rows, D, generator=sc.gen(3)).to(sc.DT[dtype])
    x[:, ::5] = 0
    w = 1 + 0.2 * torch.randn(D, generator=sc.gen(4))
    w[:group] *= tiny
    _, _, q, scale = binding.ida_rmsnorm(x.cuda(), w.cuda(), group=group)
    torch.cuda.synchronize()
    assert binding.ida_device_error() == 0
    y = orc.rmsnorm(x.double(), w.double(), 1e-6)
    top = y.reshape(rows, -1, group).abs().amax(-1)
    assert bool((scale > 0).all())
    assert worst(scale, top / 448, 64 * U32 * top / 448 + 2.0 ** -149) <= 1
    s = scale.cpu().double().repeat_interleave(group, -1)
    got = q.float().cpu().double()
    assert bool(torch.isfinite(got).all()) and not got[:, ::5].any()
    assert worst(got * s, y, (2.0 ** -4 + 128 * U32) * y.abs() + 2.0 ** -10 * s + 2.0 ** -149) <= 1
