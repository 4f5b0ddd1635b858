"""The feed-forward block and the 8-bit calls for a few rows, as decoding makes them."""
import pytest
import torch

from linear_token_mixer_sc_gb300 import binding
from tests import ffn_cases as fc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 8])
@pytest.mark.parametrize("captured", [False, True])
def test_weights_written_just_before_a_call(T, dtype, captured):
    """Every input is rewritten between calls, each by a kernel or a copy directly before them: no call reads what lay there
    before, whichever of its launches reads early."""
    D, F = 1024, 2048
    sets = [[t.cuda() for t in (fc.rows(T, D, dtype, 10 * i), *fc.weights(D, F, dtype, 10 * i + 1))] for i in range(3)]
    want = [binding.ida_ffn(*s)[0].clone() for s in sets]
    on, outs = [torch.empty_like(t) for t in sets[0]], [torch.empty_like(want[0]) for _ in sets]

    def calls():
        for s, out in zip(sets, outs):
            for k in (3, 0, 1, 2):  # w_down first, or behind the others
                on[k].copy_(s[k])
            binding.ida_ffn(*on, out=out)
        for s, out in zip(sets, outs):
            for k in (0, 1, 2, 3):
                torch.mul(s[k], 1, out=on[k])
            again = binding.ida_ffn(*on)[0]
            out.copy_(torch.where(again == out, again, torch.nan))

    if captured:
        calls()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            calls()
        for t in (*on, *outs):
            t.fill_(torch.nan)
        graph.replay()
    else:
        for _ in range(20):
            calls()
    torch.cuda.synchronize()
    assert binding.ida_device_error() == 0
    for out, w in zip(outs, want):
        assert torch.equal(out, w)


@pytest.mark.parametrize("T", [1, 3, 8])
def test_a_product_beyond_bf16(T):
    """h = g u between the largest bf16 number and the largest fp32 one, in a call of few rows, which keeps it in two parts."""
    x, w, wd = torch.zeros(T, 16), torch.zeros(2, 24, 16), torch.zeros(16, 24)
    x[:, 0] = 1
    w[0, :, 0], w[1, :, 0], wd[:] = 181 * 2.0 ** 56, 181 * 2.0 ** 57, 2.0 ** -70
    w[1, 1::2, 0] *= -0.5
    args = [t.bfloat16().cuda() for t in (x, *w, wd)]
    out, acts = binding.ida_ffn(*args, acts=True)
    g, u = (x.double() @ t.double().t() for t in w)
    h = g * u
    assert float(h.abs().max()) < torch.finfo(torch.float32).max and not bool(torch.isfinite(h.bfloat16()).all())
    want = h @ wd.double().t()
    # two parts leave 2^-16 of each product; the output is rounded
    bound = 2.0 ** -15 * (h.abs() @ wd.double().abs().t()) + 2.0 ** -8 * want.abs()
    assert bool(((out.cpu().double() - want).abs() <= bound).all())
    assert torch.equal(acts[2].cpu(), h.bfloat16())
