"""svq_paged_attention's logarithms where they are small: few keys and small scores.

Bar, with S = scale * sum |q k| of the largest score, in u = 2^-24: the products' sum in head_dim / 16 steps, each off
by 4 u of S at most (the tensor cores may cut), its two chains' sum and the scaling by log2 e, itself rounded, 3 u; the
way back, ln 2 rounded and one fused addition, 2 u of the logarithm.  One key: the sum of weights is 1 and its
logarithm 0, so that is all.  More keys: every weight is off by 2 u of itself (ex2), 1 u of its argument's size, which
is at most 2 S log2 e, and 1 u for each addition: their sum by (3 + keys + 6 S) u of itself at most, which the
logarithm takes over, and the logarithm's rounding 2 u of its own size, at most log(keys)."""
import math

import numpy as np
import pytest

from oracle import attention as oa
from tests import test_gpu_paged_attention as pa
from tests.gpu_util import need_gpu

import bit_spherical_vector_b200 as svq

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("kv", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("peak", [0.002, 0.05, 1.0])
@pytest.mark.parametrize("keys", [1, 2, 5])
def test_small_logarithms(keys, peak, dim, kv):
    need_gpu()
    a = pa.case(keys, [keys] * 9, 16, 2, dim, kv, peak=peak)
    svq.svq_paged_attention(**a)
    assert svq.svq_get_device_status() == svq.SVQ_OK
    c = a["cache"]
    want = oa.paged_attention(pa.f64(a["q"]), pa.f64(c.k), pa.f64(c.v), [keys] * 9, a["block_table"].cpu().numpy(),
                              float(np.float32(a["scale"])))
    got = pa.f64(a["lse"])
    for r in range(9):
        _, lse, _, size = want[r]
        tol = (4 * dim / 16 + 3) * U * size + 2 * U * np.abs(lse)
        if keys > 1:
            tol = tol + (3 + keys + 6 * size) * U + 2 * U * math.log(keys)
        assert np.all(np.abs(got[r] - lse) <= tol), (r, np.abs(got[r] - lse).max())
