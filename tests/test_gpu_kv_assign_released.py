"""svq_kv_assign with page numbers outside the pool among the pages of done requests: reported by the step that puts
them onto the free list, by whichever way it copies them, and again by the step that takes one."""
import numpy as np
import pytest

from oracle import attention as oa
from tests import test_gpu_kv_assign as ka
from tests.gpu_util import need_gpu

import bit_spherical_vector_b200 as svq

pytestmark = pytest.mark.gpu


def scene(n, width, longest, seed):
    """n requests of one-token pages, two in three done."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, n)
    lens[1] = longest
    new = np.where(np.arange(n) % 3 == 0, 1, -1)
    table = np.full((n, width), -1)
    deal = rng.permutation(int(lens.sum()) + n)
    at = 0
    for b, l in enumerate(lens):
        table[b, :l] = deal[at:at + l]
        at += l
    return lens, new, table, np.concatenate([deal[at:], np.full(at, -7)]), n


# entry by entry on one CTA and on a cluster; by runs, in the first run of a warp, its second and behind both
@pytest.mark.parametrize("n,width,longest", [(3, 30, 20), (60, 200, 90), (9, 900, 890), (9, 4000, 3990), (900, 70, 60)])
@pytest.mark.parametrize("bad", [-1, 2 ** 31 - 1, -2 ** 31, "n_pages"])
@pytest.mark.parametrize("place", ["first", "middle", "last"])
def test_bad_pages_are_reported(n, width, longest, bad, place):
    need_gpu()
    lens, new, table, free, n_free = scene(n, width, longest, n + width)
    done = [b for b in range(n) if new[b] < 0 and lens[b] > 1]
    b = {"first": done[0], "middle": done[len(done) // 2], "last": done[-1]}[place]
    table[b, {"first": 0, "middle": lens[b] // 2, "last": lens[b] - 1}[place]] = free.size if bad == "n_pages" else bad
    taken = int((new > 0).sum())
    want = oa.kv_assign(lens, new, 1, table, free, n_free, taken)
    assert want is not None and svq.svq_get_device_status() == svq.SVQ_OK
    got = ka.call(lens, new, 1, table, free, n_free, taken)
    ka.same(got, want)
    assert svq.svq_get_device_status() == svq.SVQ_ERR_INVALID_ARG


def test_a_bad_page_on_the_list_is_reported_when_it_is_taken():
    need_gpu()
    table, free = np.array([[1, 900], [3, -1]]), np.array([0, -7, -7, -7])
    got = ka.call([6, 3], [-1, 0], 4, table, free, 1, 4)
    assert got["free_pages"].tolist() == [0, 1, 900, -7] and got["n_free_out"] == 3 and got["lens_out"].tolist() == [0, 3]
    assert svq.svq_get_device_status() == svq.SVQ_ERR_INVALID_ARG
    got = ka.call([0, 3], [1, 0], 4, got["block_table"], got["free_pages"], 3, 4)
    assert got["slots"].tolist() == [-1] * 4 and got["positions"].tolist() == [0, -1, -1, -1]
    assert got["n_free_out"] == 2 and got["block_table"][0, 0] == 900
    assert svq.svq_get_device_status() == svq.SVQ_ERR_INVALID_ARG


def test_good_pages_are_not():
    need_gpu()
    for n, width, longest in ((3, 30, 20), (9, 4000, 3990)):
        lens, new, table, free, n_free = scene(n, width, longest, 1)
        ka.same(ka.call(lens, new, 1, table, free, n_free, n), oa.kv_assign(lens, new, 1, table, free, n_free, n))
        assert svq.svq_get_device_status() == svq.SVQ_OK
