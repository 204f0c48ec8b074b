"""Refusals of the dense serving path beside those of test_serving_plain.py.  No GPU."""
import math

import pytest

from test_serving_plain import _packed, _tree, sala  # noqa: F401


@pytest.mark.parametrize("scale", [3e38, 2.4e38, math.inf, -1e-45])
def test_a_scale_that_is_no_number_in_log2_units_is_refused(sala, scale):  # noqa: F811
    for call in (_packed, _tree):
        assert call(sala, scale=scale) == 1
        assert b"scale" in sala.raw.sala_last_error()
