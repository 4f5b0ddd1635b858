"""Quotients and signs in e4m3, bit for bit."""
import pytest
import torch

from linear_token_mixer_sc_gb300 import binding
from tests import ffn_cases as fc
from tests.ssm_cases import DT, gen

pytestmark = pytest.mark.gpu


def _bits(q):
    return q.cpu().view(torch.uint8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_the_quantiser_keeps_signs(block_rows, dtype):
    """Zeros of either sign in blocks of zeros and beside values, and values that round to zero."""
    x = torch.randn(140, 400, generator=gen(3)).to(DT[dtype])
    x[:, 128:256] = 0
    x[torch.rand(x.shape, generator=gen(4)) < 0.2] = 0
    x[torch.rand(x.shape, generator=gen(5)) < 0.2] *= 1e-4
    x = torch.where(torch.rand(x.shape, generator=gen(6)) < 0.5, -x, x)
    assert bool((torch.signbit(x) & (x == 0)).any())
    q, scale = binding.ida_quant_e4m3(x.cuda(), rows=block_rows)
    want, wscale = fc.quantised(x, block_rows)
    assert torch.equal(scale.cpu(), wscale) and torch.equal(_bits(q), _bits(want))
