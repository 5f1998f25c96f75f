"""Rescaled rotary frequencies at the edges of their options."""

import pytest

import mixed_precision_moe_amd as mx


@pytest.mark.parametrize("scaling", [dict(kind="ramp", factor=4.0), dict(kind="bands", factor=4.0), dict(kind="bands")])
def test_a_length_that_is_missing_is_a_value_error(scaling):
    with pytest.raises(ValueError, match="length"):
        mx.rotary_frequencies(64, scaling=scaling)


@pytest.mark.parametrize("factor,want", [(0.25, 1.0), (0.99, 1.0), (1.0, 1.0), (16.0, 1.2772588722239782)])
def test_a_ramp_does_not_shrink_the_vectors_of_a_shortened_context(factor, want):
    scaling = dict(kind="ramp", factor=factor, length=8192)
    assert mx.rotary_frequencies(64, scaling=scaling)[1] == pytest.approx(want, rel=1e-15)
    assert mx.rotary_frequencies(64, scaling=dict(scaling, magnitude=0.5))[1] == 0.5


def test_a_base_of_one_has_no_pair_to_ramp_between():
    with pytest.raises(ValueError, match="base"):
        mx.rotary_frequencies(64, base=1.0, scaling=dict(kind="ramp", factor=4.0, length=8192))
