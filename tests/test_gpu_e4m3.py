"""Products of e4m3 operands with a scale for each block of 128, and their quantiser."""
import pytest
import torch

from linear_token_mixer_sc_gb300 import binding
from tests import ffn_cases as fc
from tests.ssm_cases import DT, HALF, gen, worst

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("T,K", [(1, 16), (1, 2048), (3, 144), (127, 128), (128, 256), (129, 272), (500, 1136)])
def test_quantiser(T, K, block_rows, dtype):
    x = torch.randn(T, K, generator=gen(T + K)) * torch.exp(2 * torch.randn(K, generator=gen(K)))
    x = x.to(DT[dtype])
    x[:, 16:144] = 0  # a group of zeros for some
    q, scale = binding.ida_quant_e4m3(x.cuda(), rows=block_rows)
    want, wscale = fc.quantised(x, block_rows)
    assert torch.equal(scale.cpu(), wscale)
    assert torch.equal(q.cpu().view(torch.uint8), want.view(torch.uint8))


def _operand(T, K, block_rows, seed):
    q, s = fc.quantised(torch.randn(T, K, generator=gen(seed)) * K ** -0.5, block_rows)
    return q, s * torch.exp(torch.randn(s.shape, generator=gen(seed + 1)))  # blocks of unlike size


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,N", [(1, 16, 8), (1, 2048, 264), (5, 384, 136), (8, 128, 5000), (9, 2064, 136), (17, 400, 1000), (32, 5632, 72), (33, 128, 128), (128, 144, 256), (129, 256, 264), (300, 1040, 72),
                                   (257, 640, 520), (700, 272, 1000),
                                   (33, 4112, 264), (300, 2064, 520), (500, 5632, 72), (1300, 4096, 600)])  # the last: contractions shared by pairs of SMs
def test_product(T, K, N, dtype):
    a, sa = _operand(T, K, 1, 3)
    b, sb = _operand(N, K, 128, 5)
    out = binding.ida_gemm_e4m3(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), dtype=DT[dtype])
    torch.cuda.synchronize()
    assert binding.ida_device_error() == 0
    v, e = fc.product_ref(fc.values(a, sa, 1), fc.values(b, sb, 128))
    assert worst(out, v, e + HALF[dtype] * v.abs()) <= 1


@pytest.mark.parametrize("T,D,F", [(1, 16, 16), (1, 2048, 272), (5, 384, 144), (8, 128, 1264), (9, 2064, 144), (16, 144, 128), (17, 400, 1008), (32, 2048, 80), (33, 128, 128), (128, 144, 256), (129, 256, 272), (300, 1040, 80),
                                   (700, 272, 1040)])
def test_gated_projection(T, D, F):
    a, sa = _operand(T, D, 1, 3)
    wg, sg = _operand(F, D, 128, 5)
    wu, su = _operand(F, D, 128, 7)
    q, scale = binding.ida_glu_e4m3(*[t.cuda() for t in (a, sa, wg, sg, wu, su)])
    torch.cuda.synchronize()
    assert binding.ida_device_error() == 0
    h, e = fc.glu_ref(fc.values(a, sa, 1), fc.values(wg, sg, 128), fc.values(wu, su, 128))
    blocks = -(-F // 128)
    pad = torch.zeros(T, blocks * 128, dtype=torch.float64)
    pad[:, :F] = h
    top = pad.view(T, blocks, 128).abs().amax(-1)
    pad[:, :F] = e
    etop = pad.view(T, blocks, 128).amax(-1)
    assert worst(scale, top / 448, etop / 448 + 2.0 ** -23 * top / 448) <= 1
    # a value is off by half a step of e4m3 (2^-4 of it, or half the least subnormal, 2^-10 of the scale),
    # and the quotient by a rounding of the reciprocal and one of the product
    got = fc.values(q.cpu(), scale.cpu(), 1)
    s = scale.cpu().double().repeat_interleave(128, 1)[:, :F]
    assert worst(got, h, 1.07 * e + (2.0 ** -4 + 2.0 ** -21) * h.abs() + 2.0 ** -10 * s) <= 1
