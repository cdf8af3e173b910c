"""svq_paged_attention with units that many CTAs share: row tiles of 8 and 16 query heads of every head size, joined in
one level, two and three."""
import pytest

from tests import test_gpu_paged_attention as pa
from tests.gpu_util import need_gpu, torch

pytestmark = pytest.mark.gpu
WARPS = {64: 10, 128: 8, 256: 4}


def fan(rows, dim):
    """Parts that one CTA joins at a time."""
    return 16 if dim == 64 else 32 if rows * dim <= 1024 else 16 if rows * dim <= 2048 else 8


def levels(lens, hq, hk, dim):
    """Levels of the join of the longest request's units, at least: its share of the CTAs, less the two ends."""
    rows = 8 if hq // hk <= 8 else 16
    units = hk * -(-(hq // hk) // rows)
    tiles = [-(-l // 16) for l in lens]
    ctas = min(torch.cuda.get_device_properties(0).multi_processor_count, -(-sum(tiles) * units // WARPS[dim]))
    share = max(tiles) * ctas // (sum(tiles) * units) - 1
    n, at = 0, 1
    while at < share:
        at *= fan(rows, dim)
        n += 1
    return n


@pytest.mark.parametrize("peak", [1.5, 40.0])
@pytest.mark.parametrize("want,lens,hq,hk,dim,kv", [
    (1, [450, 30], 16, 1, 256, "f16"), (2, [4000, 20], 16, 1, 256, "bf16"), (3, [9000], 16, 1, 256, "f16"),
    (3, [9000], 13, 1, 256, "bf16"), (1, [2000, 700, 90], 16, 1, 128, "bf16"), (2, [9000], 16, 1, 128, "f16"),
    (2, [6000, 300], 11, 1, 128, "bf16"), (2, [4000, 4000], 32, 2, 64, "bf16"), (2, [20000, 33], 16, 1, 64, "f16"),
    (2, [9000], 4, 1, 128, "f16"), (2, [9000], 5, 1, 256, "f16"), (2, [20000], 3, 1, 64, "bf16"),
    (2, [5000, 1000], 40, 2, 256, "f16")])
def test_levels(want, lens, hq, hk, dim, kv, peak):
    need_gpu()
    assert levels(lens, hq, hk, dim) == want
    a = pa.case(hq + dim, lens, hq, hk, dim, kv, "bf16" if hq % 2 else "f16", page=32, peak=peak)
    pa.check(a)
    out, lse = a["out"].clone(), a["lse"].clone()
    for _ in range(10):
        a["out"].fill_(0)
        pa.svq.svq_paged_attention(**a)
        assert torch.equal(a["out"], out) and torch.equal(a["lse"], lse)
    assert bool((a["ws"][:65536] == 0).all())
