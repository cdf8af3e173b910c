"""svq_kv_assign with page counts next to 2^31: the largest tables and lists that the call takes."""
import pytest

from tests.gpu_util import need_gpu, torch

import bit_spherical_vector_b200 as svq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("taken", [0, 1000])
def test_releases_of_almost_all_pages(taken):
    """Three done requests give back 3 * width pages, of which a fourth takes `taken` from the top."""
    need_gpu()
    n = 4 if taken else 3
    width, n_pages = (2 ** 31 - 1) // n, 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table = torch.arange(1, n * width + 1, dtype=torch.int32, device="cuda").view(n, width)
    free = torch.full((n_pages,), -7, dtype=torch.int32, device="cuda")
    free[0] = 0
    lens, new = [width] * 3, [-1] * 3
    if taken:
        lens.append(0)
        new.append(taken)
    lens_out, n_free_out, cu = i32(*[9] * n), i32(9), i32(*[9] * (n + 1))
    pos, slots = (torch.full((1500,), 9, dtype=torch.int32, device="cuda") for _ in range(2))
    svq.svq_kv_assign(i32(*lens), i32(*new), 1, table, free, i32(1), lens_out, n_free_out, cu, pos, slots)
    assert svq.svq_get_device_status() == svq.SVQ_OK
    kept = 3 * width - taken
    assert int(n_free_out) == 1 + kept and cu.tolist() == [0] * n + [taken]
    assert lens_out.tolist() == [0] * 3 + [taken] * (n - 3)
    assert int(free[0]) == 0 and bool((free[1 + kept:] == -7).all())
    for at in range(0, kept, 1 << 28):
        end = min(kept, at + (1 << 28))
        assert torch.equal(free[1 + at:1 + end], torch.arange(at + 1, end + 1, dtype=torch.int32, device="cuda"))
    took = torch.arange(3 * width, 3 * width - taken, -1, dtype=torch.int32, device="cuda")
    assert torch.equal(slots[:taken], took) and bool((slots[taken:] == -1).all())
    assert torch.equal(pos[:taken], torch.arange(taken, dtype=torch.int32, device="cuda"))
    if taken:
        assert torch.equal(table[3, :taken], took)
