"""svq_paged_attention with infinite values in keys that count.  Every weight e^s of a finite score is positive, so an
entry with an infinite value among its v_j is that infinity, NaN beside the other sign or beside NaN, however small
the weight is; a score of -inf has weight 0, and 0 times an infinity is NaN.  All other entries and the logarithms
keep the bits that they have without the infinities."""
import numpy as np
import pytest

from tests import test_gpu_paged_attention as pa
from tests.gpu_util import need_gpu, torch

import bit_spherical_vector_b200 as svq

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def place(a, b, key):
    size = a["cache"].page_size
    return int(a["block_table"][b, key // size]), key % size


def run(a):
    b = dict(a, out=torch.full_like(a["out"], 3.0), lse=torch.full_like(a["lse"], 5.0))
    svq.svq_paged_attention(**b)
    assert svq.svq_get_device_status() == svq.SVQ_OK
    return b["out"], b["lse"]


def compare(a, planted, before):
    """planted: (request, key head, entry, value that the entry takes in every head of the group)."""
    c, (rows, hq, D) = a["cache"], a["q"].shape
    group = hq // c.n_heads
    out, lse = run(a)
    want = before[0].clone()
    column = np.arange(hq * D) if a["order"] is None else a["order"].cpu().numpy()
    for b, h, d, value in planted:
        for q in range(h * group, (h + 1) * group):
            want[b, int(column[q * D + d])] = value
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out.nan_to_num(nan=0.0, posinf=INF, neginf=-INF), want.nan_to_num(nan=0.0, posinf=INF, neginf=-INF))
    assert torch.equal(lse, before[1])


# whole units of a warp, parts joined in a CTA, parts joined by CTAs on one level and more; weights that vary by a
# factor of 2 and by far more than fp32 can hold
@pytest.mark.parametrize("peak", [0.1, 60.0])
@pytest.mark.parametrize("order", [False, True])
@pytest.mark.parametrize("lens,hq,hk,dim,kv,page", [
    ([5, 33, 16], 8, 2, 64, "f16", 16), ([5, 33, 16], 7, 1, 128, "bf16", 24), ([700, 40, 3], 8, 8, 128, "f16", 16),
    ([700, 90], 9, 1, 128, "f16", 7), ([4000, 17], 14, 2, 64, "bf16", 24), ([6000, 100], 32, 4, 128, "f16", 16),
    ([9000, 1], 16, 1, 256, "f16", 32), ([3000, 1000], 16, 2, 256, "bf16", 24), ([2000, 500], 20, 1, 64, "f16", 1)])
def test_infinite_values(lens, hq, hk, dim, kv, page, order, peak):
    need_gpu()
    a = pa.case(hq + dim, lens, hq, hk, dim, kv, "bf16" if hq % 2 else "f16", page=page, order=order, peak=peak)
    before = run(a)
    rng = np.random.default_rng(len(lens) + page)
    planted = []
    for b, n in enumerate(lens):
        for h in {0, hk - 1}:
            entries = rng.permutation(dim)[:8]
            keys = [0, n - 1, n // 2, *(int(k) for k in rng.integers(0, n, 5))]
            for d, k in zip(entries, keys):
                value = INF if rng.random() < 0.5 else -INF
                page_at, t = place(a, b, k)
                a["cache"].v[page_at, t, h, int(d)] = value
                planted.append((b, h, int(d), value))
    compare(a, planted, before)


@pytest.mark.parametrize("lens", [[200], [9000]])
@pytest.mark.parametrize("kv", ["f16", "bf16"])
def test_infinities_that_meet(lens, kv):
    """Several in one entry, near to one another and far apart: of one sign, of both, and beside NaN."""
    need_gpu()
    a = pa.case(3, lens, 4, 1, 128, kv)
    before, n = run(a), lens[0]
    planted = []
    for d, (values, result) in enumerate((([INF, INF], INF), ([-INF, -INF], -INF), ([INF, -INF], NAN), ([-INF, NAN], NAN),
                                          ([NAN, INF], NAN))):
        for far in (False, True):
            entry = 2 * d + far + 50
            for k, value in zip((3, n - 2) if far else (17, 18), values):
                page, t = place(a, 0, k)
                a["cache"].v[page, t, 0, entry] = value
            planted.append((0, 0, entry, result))
    compare(a, planted, before)


@pytest.mark.parametrize("kv", ["f16", "bf16"])
@pytest.mark.parametrize("n", [40, 5000])
def test_a_score_of_minus_infinity_weighs_nothing(n, kv):
    need_gpu()
    a = pa.case(4, [n], 4, 2, 64, kv)
    a["q"][:, :2, 7] = 0.75                                    # the first key head's queries
    a["cache"].k[place(a, 0, 21)[0], place(a, 0, 21)[1], 0, 7] = -INF
    before = run(a)
    assert bool(torch.isfinite(before[0]).all()) and bool(torch.isfinite(before[1]).all())
    page, t = place(a, 0, 21)
    a["cache"].v[page, t, 0, 5], a["cache"].v[page, t, 0, 6] = INF, -INF
    compare(a, [(0, 0, 5, NAN), (0, 0, 6, NAN)], before)


def test_rows_that_are_spoilt_whole():
    """Every value infinite, and every score NaN beside infinite values."""
    need_gpu()
    for n in (30, 3000):
        a = pa.case(5, [n], 4, 2, 64)
        a["cache"].v[:] = -INF
        out, lse = run(a)
        assert bool((out == -INF).all()) and bool(torch.isfinite(lse).all())
        a["cache"].k[place(a, 0, 9)[0], place(a, 0, 9)[1], 0, 1] = NAN
        out, lse = run(a)
        out = out.view(4, 64)
        assert bool(torch.isnan(out[:2]).all()) and bool((out[2:] == -INF).all())
        assert bool(torch.isnan(lse[0, :2]).all())
