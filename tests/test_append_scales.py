"""Scales of the 4-bit cache whose reciprocal FP32 does not hold are refused by the write,
without a GPU: rows are multiplied by RN(1 / scale), and 0 times infinity is NaN."""
import pytest

from test_attention_checks import OK, SHAPE, c_append, c_read


@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
def test_scales_without_a_reciprocal(which):
    for bad in (1e-40, 1.4e-45, 2.0 ** -129, 2.9e-39):
        assert c_append(**{which: bad}) == SHAPE, bad
        assert c_append(**{which: bad}, T=0) == SHAPE, bad
    # the least with one (1 / 2^-128 is 2^128, which rounds to infinity; 2^-127 has 2^127)
    assert c_append(**{which: 2.0 ** -128}) == SHAPE
    for good in (2.0 ** -127, 1e-30, 3e38):
        assert c_append(**{which: good}, T=0) == OK, good
    # a read multiplies: any positive scale will do
    assert c_read(**{which: 1e-40}, T=0) == OK
