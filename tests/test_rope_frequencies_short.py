"""svq_rope_frequencies (YaRN) for trained lengths so short that the fastest pairs make less than a turn."""
import math

import numpy as np
import pytest

import bit_spherical_vector_b200 as svq


@pytest.mark.parametrize("rot,base", [(16, 10000.0), (128, 1e6), (256, 1.5)])
@pytest.mark.parametrize("trained", [1, 2, 6, 7, 40, 200, 201, 5000])
def test_pairs_below_one_turn_are_divided_by_the_scale(rot, base, trained):
    plain = svq.svq_rope_frequencies(rot, base)[0]
    f, factor = svq.svq_rope_frequencies(rot, base, svq.SVQ_ROPE_YARN, 8.0, trained)
    turns = plain * trained / (2 * math.pi)
    assert factor == pytest.approx(0.1 * math.log(8.0) + 1.0, rel=1e-6)
    assert np.allclose(f[turns < 0.999], plain[turns < 0.999] / 8.0, rtol=1e-14)
    assert np.allclose(f[turns > 32.001], plain[turns > 32.001], rtol=1e-14)
    ratio = f / plain
    assert np.all(ratio <= 1.0 + 1e-15) and np.all(ratio >= 0.125 - 1e-15) and np.all(np.diff(ratio) <= 1e-15)
