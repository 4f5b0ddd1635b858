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


def _gate_exact(T, seed, size=1.0):
    """Operands whose gates are 64 and more (their sigmoid is 1) and whose products fp32 holds to a rounding each, the same
    here and there: rows' scales of 12 bits, so that products by e4m3 values often lie at a tie of e4m3 or an fp32 step
    beside it.  Returns the arguments and h in fp32."""
    F = 256
    sa = (1 + torch.randint(0, 1 << 11, (T, 1), generator=gen(seed)) / (1 << 11)).float()
    a, wg, wu = torch.zeros(T, 16), torch.zeros(F, 16), torch.zeros(F, 16)
    a[:, 0] = wg[:, 0] = 1
    v = torch.arange(8, 16) * 2.0 ** torch.randint(-9, 3, (F // 8, 1), generator=gen(seed + 1))
    v[:, ::2] *= -1
    wu[:, 0] = v.flatten()
    wu[0::128, 0], wu[5, 0] = torch.tensor([64.0, 56.0]), 0
    one = torch.ones(2, 1)
    h = (64 * sa) * (wu[:, 0] * (sa * size))
    return [t.cuda() for t in (a.to(fc.E4M3), sa, wg.to(fc.E4M3), 64 * one, wu.to(fc.E4M3), size * one)], h


@pytest.mark.parametrize("T,times", [(8, 100), (3000, 1)])
def test_the_gate_quantises_as_the_quantiser(T, times):
    for seed in range(times):
        args, h = _gate_exact(T, 10 * seed)
        q, scale = binding.ida_glu_e4m3(*args)
        want, wscale = binding.ida_quant_e4m3(h.cuda())
        assert torch.equal(scale, wscale)
        assert torch.equal(_bits(q), _bits(want)), int((_bits(q) != _bits(want)).sum())


@pytest.mark.parametrize("T", [8, 3000])
@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -138, 2.0 ** 100])
def test_the_gate_quantises_products_of_any_size(T, size):
    """Scales down to subnormal ones: every factor is a rounding of fp32's, here and there."""
    args, h = _gate_exact(T, 5, size)
    q, scale = binding.ida_glu_e4m3(*args)
    want, wscale = binding.ida_quant_e4m3(h.cuda())
    assert torch.equal(scale, wscale) and bool((scale > 0).all())
    assert torch.equal(_bits(q), _bits(want))
