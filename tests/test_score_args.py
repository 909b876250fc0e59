"""Host-only checks of the arguments of attention with changed scores, beside test_score_abi.py."""
import ctypes
import math

import pytest

from exact_io_aware_83_b200 import fa


@pytest.mark.parametrize("cap", [5e-324, 1e-50, 1e-42, 1e-30, 30.0, 1e30, 3.4e38, 1e39, 1e300])
def test_positive_caps_stay_positive_and_finite_in_fp32(cap):
    c = ctypes.c_float(fa._cap(cap)).value
    assert c > 0.0 and math.isfinite(c)
    if 1e-30 <= cap <= 1e30:
        assert c == ctypes.c_float(cap).value


def test_other_caps_are_passed_on():
    assert fa._cap(0) == 0.0 and fa._cap(-1) == -1.0 and fa._cap(math.inf) == math.inf and math.isnan(fa._cap(math.nan))
