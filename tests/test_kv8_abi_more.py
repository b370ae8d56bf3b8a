"""Further refusals of the 8-bit cache's entry points (no GPU)."""
import pytest

from test_kv8_abi import INVALID, attention, batch, cache, lib  # noqa: F401


@pytest.mark.parametrize("scale", [2.4e38, 2.9e38, 3.4e38])
def test_scale_whose_base_two_form_overflows(lib, scale):  # noqa: F811
    assert attention(lib, batch(), cache(), scale=scale) == INVALID
