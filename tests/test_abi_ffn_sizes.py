"""Sizes that the feed-forward block's calls refuse need no workspace."""
import pytest

from linear_token_mixer_sc_gb300 import binding, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


@pytest.mark.parametrize("fn", [binding.ida_ffn_workspace_bytes, binding.ida_ffn_backward_workspace_bytes])
def test_too_many_rows(fn):
    for dtype in (0, 1):
        assert fn((1 << 28) + 1, 64, 64, dtype) == 0 and fn(1 << 27, 64, 1024, dtype) == 0 and fn(1 << 27, 1024, 64, dtype) == 0
        assert fn(1 << 28, 64, 256, dtype) > 1 << 36 and fn(1 << 26, 1024, 64, dtype) > 0
