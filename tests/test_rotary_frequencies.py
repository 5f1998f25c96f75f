"""Rescaled rotary frequencies at the edges of their options."""

import pytest

import mixed_precision_moe_amd as mx


@pytest.mark.parametrize("scaling", [dict(kind="ramp", factor=4.0), dict(kind="bands", factor=4.0), dict(kind="bands")])
def test_a_length_that_is_missing_is_a_value_error(scaling):
    with pytest.raises(ValueError, match="length"):
        mx.rotary_frequencies(64, scaling=scaling)
