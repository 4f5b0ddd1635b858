"""Arguments of the selective mixer and of the pre-norm that no kernel may see: gradients of parameters
off their element's alignment, sizes behind 2^31; and how the binding's calls take their arguments."""

import pytest
import torch

from linear_token_mixer_sc_gb300 import binding, build
from tests.test_abi_ssm_overlaps import _apart, _call

ARG = binding.IDA_ERR_ARG
no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="for machines without a CUDA device")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


@no_device
@pytest.mark.parametrize("name, outputs", [("ida_ssm_conv_backward", ("dw", "db")),
                                           ("ida_ssm_scan_backward", ("da", "dbias", "dD"))])
def test_parameter_gradients_off_their_alignment(lib, name, outputs):
    base = _apart(name)
    for k in outputs:
        for off in (1, 2, 3, 6):
            assert _call(lib, name, {**base, k: base[k] + off}) == ARG and "aligned" in binding.ida_last_error(), (k, off)
        assert _call(lib, name, {**base, k: base[k] + 4}) == binding.IDA_ERR_CUDA  # taken, but there is no device


def test_the_first_argument_by_its_name(lib):
    """Refused for what it is (a host tensor), not for how it is given."""
    x, w, b = torch.zeros(1, 8, 16), torch.zeros(16, 4), torch.zeros(16)
    p = {k: torch.zeros(1) for k in ("a_log", "dt_bias", "D")}
    scan = dict(x=x[:, :, None], b=x[:, :, None], c=x[:, :, None], dt=x[..., :1], params=p)
    calls = [(binding.ida_ssm_conv, dict(x=x, conv_w=w, conv_b=b)),
             (binding.ida_ssm_conv_backward, dict(x=x, dout=x, conv_w=w, conv_b=b)),
             (binding.ida_ssm_scan, scan), (binding.ida_ssm_scan_backward, dict(scan, dy=x[:, :, None])),
             (binding.ida_ssm_step, dict(xbc=x[0], dt=x[0, :, :1], params=p, conv_state=x, state=x, groups=1)),
             (binding.ida_rmsnorm, dict(x=x, w=b)), (binding.ida_rmsnorm_backward, dict(r=x, w=b, dy=x))]
    for fn, kw in calls:
        with pytest.raises(ValueError, match="CUDA"):
            fn(**kw)
        first = next(iter(kw))
        with pytest.raises(ValueError, match="CUDA"):
            fn(kw[first], **{k: v for k, v in kw.items() if k != first})
        with pytest.raises(TypeError, match=first):
            fn()


@pytest.mark.gpu
def test_by_name_and_on_a_stream_given_by_name(lib):
    x = torch.randn(2, 40, 64, device="cuda").bfloat16()
    w, b = torch.randn(64, 4, device="cuda"), torch.randn(64, device="cuda")
    want = binding.ida_ssm_conv(x, w, b)[0]
    norm = binding.ida_rmsnorm(x, b)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [binding.ida_ssm_conv(x=x, conv_w=w, conv_b=b)[0], binding.ida_ssm_conv(conv_b=b, x=x, stream=side, conv_w=w)[0]]
    norms = [binding.ida_rmsnorm(w=b, x=x)[0], binding.ida_rmsnorm(x=x, w=b, stream=side)[0]]
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in got) and all(torch.equal(t, norm) for t in norms)


def test_sizes_behind_31_bits(lib):
    """Sizes of 2^32 and a few do not pass for the few."""
    far = (1 << 32) + 5
    for call in (lambda: binding.ida_ssm_conv_backward_workspace_bytes(2, far, 32, 4),
                 lambda: binding.ida_ssm_scan_workspace_bytes(1, 4, far, 64, 2, 16, 1),
                 lambda: binding.ida_ssm_scan_backward_workspace_bytes(far, 4, 9, 64, 2, 16, 1),
                 lambda: binding.ida_rmsnorm_backward_workspace_bytes(far, 256)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


@pytest.mark.gpu
def test_tensors_with_sizes_behind_31_bits(lib):
    """Positions and rows that share one stored row, so that nothing large is behind them."""
    far, f = (1 << 32) + 5, dict(device="cuda")
    x, w, b = torch.zeros(1, 1, 8, **f).expand(1, far, 8), torch.zeros(8, 4, **f), torch.zeros(8, **f)
    bc, dt = x.unsqueeze(2), x[..., :1]
    p = {"a_log": b[:1], "dt_bias": b[:1], "D": b[:1]}
    for call in (lambda: binding.ida_ssm_conv(x, w, b), lambda: binding.ida_ssm_conv_backward(x, x, w, b),
                 lambda: binding.ida_ssm_scan(bc, bc, bc, dt, p), lambda: binding.ida_ssm_scan_backward(bc, bc, bc, dt, p, bc),
                 lambda: binding.ida_ssm_step(x[0], dt[0], {**p, "conv_w": w, "conv_b": b}, w, w[:, :, None, None], 1)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


@pytest.mark.gpu
def test_as_many_rows_as_an_int_counts(lib):
    """2^31 - 1 rows of 8 channels: the last ones' norms, and a row more is refused."""
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 70 GB")
    rows = (1 << 31) - 1
    store = torch.zeros(rows + 1, 8, dtype=torch.bfloat16, device="cuda")
    x, w = store[:rows], torch.ones(8, device="cuda")
    x[-3:] = torch.arange(24, device="cuda").view(3, 8) - 7
    out = binding.ida_rmsnorm(x, w)[0]
    assert torch.equal(out[-3:], binding.ida_rmsnorm(x[-3:].clone(), w)[0]) and not out[:9].any() and not out[rows - 9:-3].any()
    del out
    with pytest.raises(ValueError, match="2\\^31"):
        binding.ida_rmsnorm(store, w)
