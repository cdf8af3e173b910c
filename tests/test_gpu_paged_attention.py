"""GPU parity of svq_paged_attention with the fp64 oracle.

Bar for each entry of o: half a step of the output type at the exact value, plus (2 d + a) S with S = sum_j p_j |v_j|.
  d: error of a score.  The products of a head are exact and summed in fp32 in head_dim / 16 steps, each off by at
     most 2 u' of what it adds (u' = 2^-23: the tensor cores may cut instead of rounding): (head_dim / 16 + 2) 2^-22
     of scale * sum |q k|, its largest over the keys; the scaling adds 2^-23 of the same.
  a: everything after the scores: the exponential (2^-22 and 2^-22 of its argument's rounding, counted in d for
     arguments up to d's size, else below 2^-24 * 40), the two-term weight (2^-17 for bf16, 2^-21 for fp16), one
     fp32 accumulation per tile of 16 keys (2^-22 each) and one rescaling per new maximum (2^-23, at most one a
     tile), the joins: (2 * tiles + 64) 2^-22 + 2^-16 (bf16) or 2^-20 (fp16).
lse: d + a + 2^-22 |lse|."""
import math

import numpy as np
import pytest

import synth
from oracle import attention as oa
from tests.gpu_util import need_gpu, torch

import bit_spherical_vector_b200 as svq

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


def f64(t):
    return t.detach().float().cpu().double().numpy()


def workspace(cache, heads):
    ws = torch.full((svq.svq_paged_attention_workspace_size(cache, heads),), 255, dtype=torch.uint8, device="cuda")
    ws[:65536] = 0                                            # the counters; the rest may hold anything
    return ws


def case(seed, lens, hq, hk, dim, kv="f16", out="f16", page=16, layout="nhd", rows=None, cu=None, lse=True, order=False,
         peak=1.5, spare=2, width=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    n = len(lens)
    used = [-(-l // page) for l in lens]
    n_pages = sum(used) + spare
    # everything that belongs to no token is NaN
    shape = (n_pages, hk, page, dim) if layout == "hnd" else (n_pages, page, hk, dim)
    k, v = (torch.full(shape, float("nan"), dtype=DT[kv], device="cuda") for _ in range(2))
    if layout == "hnd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    width = width or max(1, max(used))
    table = np.full((n, width), -5)
    deal = rng.permutation(n_pages)
    at = 0
    for b, l in enumerate(lens):
        table[b, :used[b]] = deal[at:at + used[b]]
        at += used[b]
        for j in range(used[b]):
            c = min(page, l - j * page)
            p = int(table[b, j])
            k[p, :c] = torch.randn((c, hk, dim), generator=g, device="cuda").to(DT[kv])
            v[p, :c] = (torch.randn((c, hk, dim), generator=g, device="cuda") + 0.25).to(DT[kv])
    rows = n if rows is None else rows
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
    perm = rng.permutation(hq * dim)
    cache = svq.KvCache(k, v)
    return dict(q=(peak * torch.randn((rows, hq, dim), generator=g, device="cuda")).to(DT[kv]), cache=cache, lens=i32(lens),
                block_table=i32(table), scale=1 / math.sqrt(dim),
                out=torch.full((rows, hq * dim), 3.0, dtype=DT[out], device="cuda"), ws=workspace(cache, hq),
                cu_rows=None if cu is None else i32(cu), order=i32(perm) if order else None,
                lse=torch.full((rows, hq), 5.0, device="cuda") if lse else None)


def check(a, run=True, status=svq.SVQ_OK):
    c = a["cache"]
    rows, hq, D = a["q"].shape
    if run:
        svq.svq_paged_attention(**a)
        assert svq.svq_get_device_status() == status
    out = f64(a["out"])
    if a["order"] is not None:
        out = out[:, a["order"].cpu().numpy()]
    out = out.reshape(rows, hq, D)
    cu = None if a["cu_rows"] is None else a["cu_rows"].cpu().numpy()
    lens = np.clip(a["lens"].cpu().numpy(), 0, a["block_table"].shape[1] * c.page_size)
    want = oa.paged_attention(f64(a["q"]), f64(c.k), f64(c.v), lens, a["block_table"].cpu().numpy(),
                              float(np.float32(a["scale"])), cu)
    eps = torch.finfo(a["out"].dtype).eps
    tiles = -(-int(max(lens)) // 16)
    acc = (2 * tiles + 64) * 2.0 ** -22 + (2.0 ** -16 if c.dtype is torch.bfloat16 else 2.0 ** -20)
    for r in range(rows):
        if r not in want:                                     # rows of nobody are left alone
            assert np.all(out[r] == 3.0)
            assert a["lse"] is None or bool((a["lse"][r] == 5.0).all())
            continue
        o, lse, size, score = want[r]
        d = ((D / 16 + 2) * 2.0 ** -22 + 2.0 ** -23) * score + 40 * 2.0 ** -24
        err = (2 * d[:, None] + acc) * size
        tol = eps / 2 * (np.abs(o) + err) + err + TINY[a["out"].dtype] / 2
        off = np.abs(out[r] - o) - tol
        assert off.max() <= 0, (r, np.unravel_index(off.argmax(), off.shape), off.max())
        if a["lse"] is not None:
            got = f64(a["lse"][r])
            fin = np.isfinite(lse)
            assert np.array_equal(np.isfinite(got), fin) and np.all(got[~fin] == -np.inf)
            assert np.all(np.abs(got[fin] - lse[fin]) <= (d + acc)[fin] + 2.0 ** -22 * np.abs(lse[fin]))


@pytest.mark.parametrize("kv", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,dim", [(1, 1, 64), (8, 8, 64), (32, 8, 128), (32, 4, 128), (14, 2, 64), (3, 1, 256),
                                       (9, 1, 128), (16, 1, 256), (24, 2, 128), (17, 1, 64), (40, 2, 256), (80, 1, 64)])
def test_types_and_head_layouts(hq, hk, dim, kv):
    need_gpu()
    check(case(hq + dim, [1, 77, 16, 0, 33], hq, hk, dim, kv, "bf16" if hq % 2 else "f16", page=16 if hk > 1 else 24,
               layout="hnd" if hq > 16 else "nhd", order=hq % 3 == 0))


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 32, 127, 128, 129, 255, 257, 1000, 2049, 5000])
@pytest.mark.parametrize("page", [16, 7])
def test_one_request_of_every_length(length, page):
    need_gpu()
    check(case(length, [length], 8, 2, 128, page=page))


@pytest.mark.parametrize("page,layout", [(1, "nhd"), (3, "hnd"), (8, "nhd"), (24, "hnd"), (32, "nhd"), (64, "hnd"),
                                         (128, "nhd"), (1000, "hnd")])
def test_pages(page, layout):
    need_gpu()
    check(case(page, [1, 100, 999, 0, 48, 24, 500], 12, 3, 128, page=page, layout=layout, out="bf16"))


@pytest.mark.parametrize("seed", range(4))
def test_many_ragged_requests(seed):
    """More units than warps, fewer, and single requests far longer than the others."""
    need_gpu()
    rng = np.random.default_rng(seed)
    lens = [int(x) for x in rng.integers(0, [40, 200, 30, 700][seed], [300, 60, 1500, 9][seed])]
    lens[len(lens) // 3] = 6000
    check(case(seed, lens, [4, 16, 2, 6][seed], [2, 2, 1, 3][seed], [64, 128, 64, 256][seed], "bf16" if seed % 2 else "f16",
               page=16))


@pytest.mark.parametrize("hq,dim", [(16, 64), (16, 128), (16, 256), (2, 128)])
def test_most_requests(hq, dim):
    need_gpu()
    lens = np.random.default_rng(dim).integers(0, 30, 4096)
    lens[4095] = 700
    check(case(hq, [int(l) for l in lens], hq, 1, dim))


def test_rows_of_a_step():
    """Requests without a row are left out, a request's query is its last row of the step, other rows keep what
    they held."""
    need_gpu()
    check(case(1, [50, 60, 0, 70, 80, 5], 8, 2, 128, rows=9, cu=[0, 3, 3, 4, 5, 5, 7], order=True))


def test_nothing_but_empty_requests():
    need_gpu()
    check(case(2, [0, 0, 0], 8, 2, 64))
    a = case(3, [0, 7], 8, 2, 64, rows=2, cu=[0, 0, 0])
    check(a)


def test_sharp_scores_and_ties():
    """Scores hundreds apart, all keys alike, and one key far ahead of 5000 others that hold most of the sum."""
    need_gpu()
    check(case(4, [300, 2000], 8, 2, 128, peak=60.0))
    a = case(5, [333], 8, 2, 128)
    a["cache"].k[:] = a["cache"].k[int(a["block_table"][0, 0]), 0]
    check(a)
    for kv in ("f16", "bf16"):
        a = case(6, [5000], 4, 1, 64, kv=kv, peak=0.05)
        # a sink: the first key scores 13 above the rest, whose sum is then about 1 % of it
        q = torch.full_like(a["q"], 0.25)
        a["q"].copy_(q + a["q"])
        p0 = int(a["block_table"][0, 0])
        a["cache"].k[p0, 0] = 13.0 / (0.25 * 64 * a["scale"])
        a["cache"].v[p0, 0] = 0.0
        check(a)


def test_infinities_and_nan_behind_the_length():
    """Every entry that belongs to no token holds NaN in all cases here; this one plants infinities as well, and a
    table that names no page behind the length."""
    need_gpu()
    a = case(7, [17, 250], 8, 2, 128, page=24)
    for b, l in ((0, 17), (1, 250)):
        p = int(a["block_table"][b, l // 24])
        a["cache"].k[p, l % 24:] = float("inf")
        a["cache"].v[p, l % 24:] = float("-inf")
    a["block_table"][0, 1:] = 2 ** 31 - 1
    check(a)


def test_nan_in_a_key_that_counts_is_seen():
    need_gpu()
    a = case(8, [40, 40], 4, 2, 64)
    a["cache"].k[int(a["block_table"][0, 1]), 3, 0, 5] = float("nan")
    svq.svq_paged_attention(**a)
    out = a["out"].view(2, 4, 64)
    assert bool(torch.isnan(out[0, :2]).all()) and bool(torch.isfinite(out[0, 2:]).all())
    assert bool(torch.isfinite(out[1]).all())
    for lens in ([40], [4000]):                                # nothing but NaN, whole and joined
        a = case(8, lens, 4, 2, 64)
        a["cache"].k.fill_(float("nan"))
        svq.svq_paged_attention(**a)
        assert bool(torch.isnan(a["out"]).all()) and bool(torch.isnan(a["lse"]).all())


def test_bad_pages_lengths_rows_and_columns():
    need_gpu()
    a = case(9, [100, 50, 30], 8, 2, 64)
    a["block_table"][0, 2] = a["cache"].n_pages
    a["block_table"][1, 0] = -1
    a["block_table"][2, :2] = 2 ** 31 - 1                      # a request with no key left
    check(a, status=svq.SVQ_ERR_INVALID_ARG)
    b = case(10, [100, 50], 8, 2, 64)
    full = int(b["block_table"].shape[1]) * 16                 # 112: seven pages, the last twelve keys' NaN
    b["lens"][0], b["lens"][1] = 10 ** 6, -4
    b["cache"].k.nan_to_num_(0.5)
    b["cache"].v.nan_to_num_(0.5)
    assert full == 112
    check(b, status=svq.SVQ_ERR_INVALID_ARG)
    c = case(11, [20, 30, 40], 4, 2, 64, rows=2, cu=[0, 1, 2, 3])
    svq.svq_paged_attention(**c)
    assert svq.svq_get_device_status() == svq.SVQ_ERR_INVALID_ARG
    check(dict(c, lens=c["lens"][:2].clone(), block_table=c["block_table"][:2].clone(), cu_rows=c["cu_rows"][:3].clone()),
          run=False)
    for lens in ([20, 30], [2000, 30]):                        # whole units and joined ones
        d = case(12, lens, 4, 2, 64, order=True)
        gone = int(d["order"][7])
        d["order"][7] = 4 * 64
        svq.svq_paged_attention(**d)
        assert svq.svq_get_device_status() == svq.SVQ_ERR_INVALID_ARG
        assert bool((d["out"][:, gone] == 0.0).all()) and not bool((d["out"] == 3.0).any())


def test_pool_beyond_32_bit_offsets():
    need_gpu()
    page, hk, dim = 64, 8, 128
    n_pages = (1 << 31) // (page * hk * dim) + 4
    a = case(13, [200, 130], 16, hk, dim, page=page)
    k = torch.empty((n_pages, page, hk, dim), dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    move = {p: n_pages - 1 - p for p in range(a["cache"].n_pages)}
    table = a["block_table"].cpu().numpy().copy()
    for p, t in move.items():
        k[t], v[t] = a["cache"].k[p], a["cache"].v[p]
    for b in range(2):
        for j in range(table.shape[1]):
            table[b, j] = move.get(int(table[b, j]), -1)
    svq.svq_paged_attention(**a)
    b = dict(a, cache=svq.KvCache(k, v), block_table=torch.from_numpy(table).cuda(), out=torch.zeros_like(a["out"]),
             lse=torch.zeros_like(a["lse"]))
    svq.svq_paged_attention(**b)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


def test_same_results_run_after_run_and_counters_left_at_zero():
    need_gpu()
    a = case(14, [3000, 10, 700], 8, 2, 128)
    svq.svq_paged_attention(**a)
    first = a["out"].clone()
    for _ in range(20):
        a["out"].fill_(0)
        svq.svq_paged_attention(**a)
        assert torch.equal(a["out"], first)
    assert bool((a["ws"][:65536] == 0).all())


def test_one_workspace_for_gemv_and_attention():
    """A GEMV with shared row tiles and attention calls of other shapes, in turn on one workspace."""
    need_gpu()
    m = synth.make_matrix(3, 3, 2560, 9728, 8)
    W = svq.SvqWeight.from_synth(m)
    x = torch.randn((1, 9728), device="cuda").half()
    y0, y1 = (torch.empty((1, 2560), device="cuda") for _ in range(2))
    a, b = case(15, [4000], 8, 2, 128), case(16, [100, 900], 16, 1, 64)
    nb = max(svq.svq_linear_gemv_workspace_size(W, 1), a["ws"].numel(), b["ws"].numel())
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    svq.svq_workspace_init(ws)
    svq.svq_linear_gemv(W, x, y0, ws)
    for c in (a, b, a, b):
        c["ws"] = ws
        svq.svq_paged_attention(**c)
        svq.svq_linear_gemv(W, x, y1, ws)
        assert torch.equal(y0, y1)
    check(a, run=False)
    check(b, run=False)


def test_captured_call_follows_the_lengths():
    """One captured call, replayed while the requests grow: the split is made anew on the device."""
    need_gpu()
    a = case(17, [1200, 3, 640], 8, 2, 128)
    a["lens"][:] = 1
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        svq.svq_paged_attention(**a)
    for lens in ([1, 1, 1], [1200, 3, 640], [0, 2, 5], [900, 0, 0]):
        a["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        a["out"].fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        check(a, run=False)


def test_two_streams_with_their_own_workspaces():
    need_gpu()
    cases = [case(18 + i, [2500, 40], 8, 2, 128) for i in range(2)]
    for c in cases:
        svq.svq_paged_attention(**c)
    want = [c["out"].clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(cases, streams):
            svq.svq_paged_attention(**c, stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert torch.equal(c["out"], w)


def test_refusals_and_binding_checks():
    need_gpu()
    a = case(20, [20, 30], 8, 2, 64, order=True)
    short = a["ws"][:a["ws"].numel() - 1]
    for bad, status in ((dict(ws=short), svq.SVQ_ERR_WORKSPACE), (dict(ws=a["ws"][8:]), svq.SVQ_ERR_WORKSPACE),
                        (dict(scale=float("nan")), svq.SVQ_ERR_INVALID_ARG)):
        with pytest.raises(svq.SvqError) as e:
            svq.svq_paged_attention(**{**a, **bad})
        assert e.value.status == status
    with pytest.raises(svq.SvqError):
        svq.svq_paged_attention(**{**a, "q": torch.zeros((2, 7, 64), dtype=torch.float16, device="cuda"), "order": None,
                                   "out": torch.zeros((2, 448), dtype=torch.float16, device="cuda"), "lse": None})
    for bad in (dict(q=a["q"].bfloat16()), dict(q=a["q"][:1]), dict(out=a["out"][:, :256]), dict(lens=a["lens"].long()),
                dict(block_table=a["block_table"][:1]), dict(block_table=a["block_table"].repeat(1, 2)[:, ::2]),
                dict(order=a["order"][:5]), dict(lse=a["lse"].double()), dict(lse=a["lse"][:, :4]), dict(lens=a["lens"].cpu()),
                dict(cu_rows=a["lens"]), dict(q=a["q"].transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            svq.svq_paged_attention(**{**a, **bad})
    assert bool((a["out"] == 3.0).all())
