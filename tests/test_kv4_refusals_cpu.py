"""Refusals of the 4-bit attention before any launch, without a GPU."""
import pytest

from tests.test_kv4_cpu import _attn, lib  # noqa: F401


@pytest.mark.parametrize("scale", [3e38, -3e38, float("inf"), float("nan")])
def test_scales_that_are_not_finite_in_float32(lib, scale):  # noqa: F811
    """Scores are taken in units of log 2: 1.44 times the scale has to be finite too."""
    assert _attn(lib, scale=scale) == -3
