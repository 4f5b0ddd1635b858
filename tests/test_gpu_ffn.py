"""The gated feed-forward block and its gradients against 64 bits."""
import pytest
import torch

from linear_token_mixer_sc_gb300 import binding
from tests import ffn_cases as fc
from tests.ssm_cases import DT, worst

pytestmark = pytest.mark.gpu

# rows, channels, hidden channels: one row, tiles that end anywhere, contractions shorter than a block
SIZES = [(1, 8, 8), (1, 64, 176), (2, 128, 344), (7, 40, 24), (8, 2048, 5632), (9, 264, 520), (16, 72, 1000), (31, 200, 72), (33, 64, 64), (128, 64, 128), (129, 72, 136), (251, 64, 176),
         (256, 256, 256), (300, 520, 264), (513, 768, 520), (1000, 136, 1032),
         (40, 72, 2056), (40, 1024, 3328), (300, 264, 2304), (1500, 520, 1096), (2100, 64, 72)]  # contractions shared by pairs of SMs


def _inputs(T, D, F, dtype, seed=0):
    return (fc.rows(T, D, dtype, seed), *fc.weights(D, F, dtype, seed + 1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,F", SIZES)
def test_forward(T, D, F, dtype):
    x, wg, wu, wd = _inputs(T, D, F, dtype)
    ref = fc.forward_ref(x, wg, wu, wd, dtype)
    on = [t.cuda() for t in (x, wg, wu, wd)]
    out, acts = binding.ida_ffn(*on, acts=True)
    alone, none = binding.ida_ffn(*on)
    torch.cuda.synchronize()
    assert binding.ida_device_error() == 0 and none is None
    for name, got in zip(("out", "g", "u", "h"), (out, *acts)):
        assert worst(got, *ref[name]) <= 1, name
    assert worst(alone, *ref["out"]) <= 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,F", SIZES)
def test_backward(T, D, F, dtype):
    x, wg, wu, wd = _inputs(T, D, F, dtype)
    dy = fc.rows(T, D, dtype, 7)
    ref = fc.forward_ref(x, wg, wu, wd, dtype)
    acts = torch.stack([ref[k][0] for k in "guh"]).to(DT[dtype])
    want = fc.backward_ref(x, wg, wu, wd, acts, dy, dtype)
    got = binding.ida_ffn_backward(*[t.cuda() for t in (x, wg, wu, wd, acts, dy)])
    torch.cuda.synchronize()
    assert binding.ida_device_error() == 0
    for name, (v, e) in want.items():
        assert worst(got[name], v, e) <= 1, name
