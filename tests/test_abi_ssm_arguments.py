"""Arguments of the selective mixer and of the pre-norm that no kernel may see: gradients of parameters
off their element's alignment."""

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
