"""The 8-bit gate's arithmetic, through the scales that it writes in fp32."""
import pytest
import torch

from linear_token_mixer_sc_gb300 import binding
from tests import ffn_cases as fc
from tests.ssm_cases import gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [8, 1 << 17])
def test_sigmoid(T):
    """Rows whose product has one channel: with a gate -m, u = m and values of 1 its scale is m^2 sigmoid(-m) / 448.  The sigmoid
    is off by (m + 8) 2^-24: half a step of m log2 e, 2^-24 of it; the exponential's 2^-22; half a step of the
    addition; the reciprocal's 2^-23.  Then come two products and a division, 2^-24 each.  The half step counts
    most where m log2 e lies just above a power of two: above 11.1, 22.2 and 44.4."""
    for low in (11.09, 22.19, 44.37, 60.0, 86.0):
        m = low + 0.3 * torch.rand(T, generator=gen(int(low)))
        a, w = torch.zeros(T, 16), torch.zeros(16, 16)
        a[:, 0] = w[0, 0] = 1
        one = torch.ones(1, 1).cuda()
        q, scale = binding.ida_glu_e4m3(a.to(fc.E4M3).cuda(), m[:, None].cuda(), (-w).to(fc.E4M3).cuda(), one, w.to(fc.E4M3).cuda(), one)
        torch.cuda.synchronize()
        want = m.double() ** 2 * torch.sigmoid(-m.double()) / 448
        rel = (scale[:, 0].cpu().double() / want - 1).abs()
        assert bool((rel <= (m.double() + 11) * 2.0 ** -24).all()), (low, float((rel * 2 ** 24).max()))
        assert bool((q.float()[:, 0] == -448).all()) and bool((q.float()[:, 1:] == 0).all())
