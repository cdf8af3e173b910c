"""GPU parity of svq_kv_assign with the oracle's step-by-step bookkeeping: every output equal, entry for entry."""
import numpy as np
import pytest

from oracle import attention as oa
from tests.gpu_util import need_gpu, torch

import bit_spherical_vector_b200 as svq

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def scene(rng, n, page, longest, rows, done=0.15, idle=0.15, prompts=0.2, spare=3):
    """Lengths, new counts, a table of distinct pages and the list of the others."""
    lens = rng.integers(0, longest + 1, n)
    new = np.ones(n, np.int64)
    pick = rng.random(n)
    new[pick < prompts] = rng.integers(1, max(2, rows // max(1, int(n * prompts) + 1)), (pick < prompts).sum())
    new[(pick >= prompts) & (pick < prompts + done)] = -rng.integers(1, 9)
    new[(pick >= prompts + done) & (pick < prompts + done + idle)] = 0
    while np.maximum(new, 0).sum() > rows:
        new[np.argmax(new)] = 0
    held = -(-lens // page)
    width = int(max(1, -(-(lens + np.maximum(new, 0)).max() // page)))
    n_pages = int(held.sum() + np.maximum(-(-(lens + np.maximum(new, 0)) // page) - held, 0).sum() + spare)
    deal = rng.permutation(n_pages)
    table = np.full((n, width), -1)
    at = 0
    for b in range(n):
        table[b, :held[b]] = deal[at:at + held[b]]
        at += held[b]
    free = np.full(n_pages, -7)
    free[:n_pages - at] = deal[at:]
    return lens, new, table, free, n_pages - at


def call(lens, new, page, table, free, n_free, rows, in_place=False):
    t = {"lens": dev(lens), "table": dev(table), "free": dev(free), "n_free": dev([n_free])}
    out = {k: torch.full((m,), -99, dtype=torch.int32, device="cuda")
           for k, m in (("cu", len(lens) + 1), ("pos", rows), ("slots", rows))}
    lens_out = t["lens"] if in_place else torch.full((len(lens),), -99, dtype=torch.int32, device="cuda")
    nf_out = t["n_free"] if in_place else torch.full((1,), -99, dtype=torch.int32, device="cuda")
    svq.svq_kv_assign(t["lens"], dev(new), page, t["table"], t["free"], t["n_free"], lens_out, nf_out, out["cu"],
                      out["pos"], out["slots"])
    torch.cuda.synchronize()
    n = lambda x: x.cpu().numpy()
    return {"block_table": n(t["table"]), "free_pages": n(t["free"]), "lens_out": n(lens_out),
            "n_free_out": int(nf_out[0]), "cu_rows": n(out["cu"]), "positions": n(out["pos"]), "slots": n(out["slots"])}


def same(got, want):
    for k, v in want.items():
        assert np.array_equal(got[k], v), k


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,page,longest,rows", [
    (1, 16, 0, 1), (1, 1, 40, 5), (3, 16, 100, 3), (16, 16, 4000, 16), (17, 24, 700, 333), (64, 3, 50, 4096),
    (100, 32, 9000, 4097), (511, 16, 300, 600), (513, 8, 64, 20000), (1500, 64, 4000, 9001), (4096, 16, 200, 8192)])
def test_against_oracle(n, page, longest, rows, in_place):
    need_gpu()
    rng = np.random.default_rng(n * 7 + page + rows)
    lens, new, table, free, n_free = scene(rng, n, page, longest, rows)
    want = oa.kv_assign(lens, new, page, table, free, n_free, rows)
    assert want is not None
    same(call(lens, new, page, table, free, n_free, rows, in_place), want)
    assert svq.svq_get_device_status() == svq.SVQ_OK


# rows of done requests that are kept free: many short ones, a few long ones, long ones between short ones
@pytest.mark.parametrize("n,longest,rows", [(4096, 90, 100), (40, 9000, 50), (3000, 250, 16000), (7, 60000, 9000)])
@pytest.mark.parametrize("mixed", [False, True])
def test_long_releases(n, longest, rows, mixed):
    need_gpu()
    rng = np.random.default_rng(n + longest)
    lens, new, table, free, n_free = scene(rng, n, 1, longest, rows, done=0.6, spare=11)
    new[n // 2] = -1                                         # one done request at least, in the middle
    if mixed:
        short = rng.random(n) < 0.5
        lens[short] = np.minimum(lens[short], rng.integers(0, 3, short.sum()))
    want = oa.kv_assign(lens, new, 1, table, free, n_free, rows)
    assert want is not None
    for in_place in (False, True):
        same(call(lens, new, 1, table, free, n_free, rows, in_place), want)
    assert svq.svq_get_device_status() == svq.SVQ_OK


@pytest.mark.parametrize("last", [-1, 1, 0])
def test_long_releases_on_one_cta(last):
    need_gpu()
    rng = np.random.default_rng(3)
    lens, new = np.array([1000, 1, 0, 1000, 513, 999, 700, 1000, 900]), np.full(9, -1)
    new[-1] = last
    table = np.full((9, 910), -1)
    lens = np.minimum(lens, 910)
    deal = rng.permutation(int(lens.sum()) + 4)
    at = 0
    for b, l in enumerate(lens):
        table[b, :l] = deal[at:at + l]
        at += l
    free = np.concatenate([deal[at:], np.full(at, -7)])
    want = oa.kv_assign(lens, new, 1, table, free, 4, 5)
    assert want is not None and want["n_free_out"] > 4100
    same(call(lens, new, 1, table, free, 4, 5), want)
    assert svq.svq_get_device_status() == svq.SVQ_OK


@pytest.mark.parametrize("rows", [64, 9000])                 # one CTA and a cluster of them
@pytest.mark.parametrize("what", ["negative", "too long", "too many rows", "no pages", "free count", "huge"])
def test_refused_steps_change_nothing(what, rows):
    need_gpu()
    rng = np.random.default_rng(5)
    lens, new, table, free, n_free = scene(rng, 20, 8, 90, rows, done=0.1, spare=0)
    if what == "negative":
        lens[3] = -1
    elif what == "too long":
        lens[3], new[3] = table.shape[1] * 8, 1
    elif what == "too many rows":
        new[0] += rows + 1 - np.maximum(new, 0).sum() if new[0] >= 0 else rows + 1 - np.maximum(new, 0).sum() - new[0]
        table = np.pad(table, ((0, 0), (0, rows)), constant_values=-1)
    elif what == "no pages":
        new[new < 0] = 0
        n_free = 0
        new[0], lens[0] = 1, -(-lens[0] // 8) * 8
        table = np.pad(table, ((0, 0), (0, 2)), constant_values=0)
    elif what == "free count":
        n_free = free.size + 1
    else:
        new[:] = 2 ** 31 - 1
        lens[:] = 0
    assert oa.kv_assign(lens, new, 8, table, free, n_free, rows) is None
    got = call(lens, new, 8, table, free, n_free, rows)
    same(got, {"block_table": table, "free_pages": free, "lens_out": lens, "n_free_out": n_free,
               "cu_rows": np.zeros(21), "positions": np.full(rows, -1), "slots": np.full(rows, -1)})
    assert svq.svq_get_device_status() == svq.SVQ_ERR_INVALID_ARG


def test_pages_outside_the_pool_give_no_slot():
    need_gpu()
    table, free = np.array([[5, -1], [900, -1], [1, -1]]), np.array([0, 77, -3, 2, 3, 4])
    got = call([3, 3, 4], [1, 1, 1], 4, table, free, 2, 4)
    assert got["slots"].tolist() == [23, -1, -1, -1] and got["positions"].tolist() == [3, 3, 4, -1]
    assert got["n_free_out"] == 1 and got["lens_out"].tolist() == [4, 4, 5]
    assert svq.svq_get_device_status() == svq.SVQ_ERR_INVALID_ARG


def test_repeating_a_call_has_the_same_effect():
    need_gpu()
    rng = np.random.default_rng(9)
    lens, new, table, free, n_free = scene(rng, 40, 4, 60, 500, done=0.4)
    want = oa.kv_assign(lens, new, 4, table, free, n_free, 500)
    first = call(lens, new, 4, table, free, n_free, 500)
    same(first, want)
    same(call(lens, new, 4, first["block_table"], first["free_pages"], n_free, 500), want)


def test_captured_decode_steps_update_in_place():
    """A captured step that adds one token to every request, replayed 40 times on its own results."""
    need_gpu()
    rng = np.random.default_rng(10)
    n, page = 6, 4
    lens, _, table, free, n_free = scene(rng, n, page, 30, n, spare=100)
    table = np.pad(table, ((0, 0), (0, 12)), constant_values=-1)
    t = [dev(x) for x in (lens, np.ones(n), table, free, [n_free])]
    cu, pos, slots = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (n + 1, n, n))

    def step():
        svq.svq_kv_assign(t[0], t[1], page, t[2], t[3], t[4], t[0], t[4], cu, pos, slots)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(40):
        want = oa.kv_assign(lens, np.ones(n), page, table, free, n_free, n)
        g.replay()
        assert np.array_equal(slots.cpu().numpy(), want["slots"])
        lens, table, free, n_free = want["lens_out"], want["block_table"], want["free_pages"], want["n_free_out"]
        assert int(t[4][0]) == n_free
    assert np.array_equal(t[2].cpu().numpy(), table) and np.array_equal(t[0].cpu().numpy(), lens)


def test_binding_refuses_what_the_library_cannot_see():
    need_gpu()
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    good = dict(lens=i(2), n_new=i(2), page_size=4, block_table=i(2, 3), free_pages=i(5), n_free=i(1), lens_out=i(2),
                n_free_out=i(1), cu_rows=i(3), positions=i(4), slots=i(4))
    svq.svq_kv_assign(**good)
    for bad in (dict(n_new=i(3)), dict(block_table=i(3, 3)), dict(block_table=i(6)), dict(cu_rows=i(2)),
                dict(positions=i(3)), dict(lens=i(2).long()), dict(block_table=i(2, 6)[:, ::2]),
                dict(slots=torch.zeros(4, dtype=torch.int32)), dict(n_free=i(2))):
        with pytest.raises(ValueError):
            svq.svq_kv_assign(**{**good, **bad})
