"""GPU parity of the selective mixer where a call divides its work: sequences split into segments and
parts of them.  Each case proves from the workspace it asks for that it is divided so.

Bounds as in ``test_gpu_ssm.py``.
"""
import pytest
import torch

from linear_token_mixer_sc_gb300 import binding, build
from tests import ssm_cases as sc
from tests.ssm_cases import worst
from tests.test_gpu_ssm import _done, _on_gpu, _scan_bounds, _scan_inputs, _scan_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


# (B, N, H, d, G, M, dtype, state, fast): bf16 sequences behind 1024 positions on idle SMs
SPLIT_SCANS = [
    (1, 1100, 4, 32, 1, 16, "bf16", True, False),    # a chunk a segment
    (3, 1700, 4, 64, 2, 64, "bf16", False, False),   # segments of several chunks
    (16, 2304, 4, 8, 1, 8, "bf16", True, False),     # two segments, states of parts of them
    (1, 1300, 2, 128, 1, 128, "bf16", True, False),  # the widest tiles: one CTA an SM
    (1, 1200, 2, 256, 2, 24, "bf16", True, False),   # two slices of channels
    (2, 1500, 3, 72, 1, 72, "bf16", False, True),    # decays that underflow within a few positions
]


@pytest.mark.parametrize("case", SPLIT_SCANS, ids=str)
def test_scan_in_segments(case):
    B, N, H, d, G, M, dtype, state, _ = case
    p, row, s, C = _scan_inputs(*case)
    assert binding.ida_ssm_scan_workspace_bytes(B, H, N, d, G, M, binding.IDA_BF16) > 0
    args = (*_on_gpu(row, C, H, d, G, M), sc.cuda(p))
    given = None if s is None else s.cuda()
    y, X = binding.ida_ssm_scan(*args, state_in=given, final_state=True)
    z, none = binding.ida_ssm_scan(*args, state_in=given)
    whole = torch.empty(0, dtype=torch.uint8, device="cuda")  # no workspace: the sequence in one piece
    y1, X1 = binding.ida_ssm_scan(*args, state_in=given, final_state=True, workspace=whole)
    _done()
    ry, rX = _scan_ref(row, C, H, d, G, M, p, s)
    ya, Xa = _scan_ref(row, C, H, d, G, M, p, s, absolute=True)
    by, bX = _scan_bounds(dtype, N, ry, ya, Xa)
    for got in (y, z, y1):
        assert worst(got, ry, by) <= 1
    for got in (X, X1):
        assert worst(got, rX, bX) <= 1
    assert none is None


@pytest.mark.parametrize("case", SPLIT_SCANS[:4], ids=str)
def test_outputs_do_not_depend_on_whether_the_final_state_is_wanted(case):
    B, N, H, d, G, M = case[:6]
    p, row, s, C = _scan_inputs(*case)
    args = (*_on_gpu(row, C, H, d, G, M), sc.cuda(p))
    given = None if s is None else s.cuda()
    y, _ = binding.ida_ssm_scan(*args, state_in=given, final_state=True)
    z, _ = binding.ida_ssm_scan(*args, state_in=given)
    _done()
    assert torch.equal(y, z)
