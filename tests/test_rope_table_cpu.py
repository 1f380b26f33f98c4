"""pa_rope_table at the ends of its range of theta."""

import numpy as np
import pytest

import paged_kv_cache_352_b200 as pa


def test_theta_whose_frequencies_overflow_is_refused():
    for theta in (5e-324, 1e-310, 9e-301, 1.1e300):
        with pytest.raises(pa.PAError):
            pa.pa_rope_table(5, 128, theta)
    for theta in (1e-300, 1e300):
        assert np.isfinite(pa.pa_rope_table(2000, 128, theta)).all()
