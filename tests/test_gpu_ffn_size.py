"""Gradients of the feed-forward block where a step of their formula could pass fp32."""
import pytest
import torch

from linear_token_mixer_sc_gb300 import binding
from tests import ffn_cases as fc
from tests.ssm_cases import DT, gen, worst

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,T,D,F", [("bf16", 20, 64, 72), ("bf16", 300, 264, 520), ("f32", 20, 64, 72), ("f32", 2000, 512, 264)])
def test_closed_gates_beside_large_gradients(dtype, T, D, F):
    """Gates of -200, whose slope is 0, with up = 1e20 and dh of 1e30: dg and du are 0 or next to it, on either side of
    the rule for fp32."""
    x, wg, wu, wd = fc.rows(T, D, dtype, 1), *fc.weights(D, F, dtype, 2)
    acts = torch.randn(3, T, F, generator=gen(3))
    shut = torch.rand(T, F, generator=gen(4)) < 0.3
    acts[0][shut], acts[1][shut] = -200.0, 1e20
    dy = torch.full((T, D), 1e15)
    wd = (wd.float().abs() + 0.01) * 1e15
    open_ = ~shut
    acts[1][open_] *= 1e-30  # so that the other gradients are of usual size
    acts[0][open_] = acts[0][open_].clamp(-3, 3)
    acts, dy, wd = acts.to(DT[dtype]), dy.to(DT[dtype]), wd.to(DT[dtype])
    got = binding.ida_ffn_backward(*[t.cuda() for t in (x, wg, wu, wd, acts, dy)])
    torch.cuda.synchronize()
    want = fc.backward_ref(x, wg, wu, wd, acts, dy, dtype)
    for k in ("x", "w_gate", "w_up", "w_down"):
        assert bool(torch.isfinite(got[k]).all()), k
        assert worst(got[k], *want[k]) <= 1, k
