"""Calls of the attention step that its documentation allows beside the usual ones: pools in other orders, more rows
than requests, steps without rows, positions below zero, a captured call before any other of the process."""
import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import attention as oa
from tests import test_gpu_kv_assign as ka
from tests import test_gpu_paged_attention as pa
from tests import test_gpu_rope_cache as rc
from tests.gpu_util import need_gpu, torch

import bit_spherical_vector_b200 as svq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("order", ["interleaved", "heads first", "gaps"])
@pytest.mark.parametrize("page", [16, 24, 1])
def test_pools_in_other_orders(order, page):
    need_gpu()
    a = pa.case(page, [50, 0, 700], 6, 3, 128, page=page)
    c = a["cache"]
    n, hk, D = c.n_pages, 3, 128
    nan = lambda *s: torch.full(s, float("nan"), dtype=torch.float16, device="cuda")
    if order == "interleaved":
        pool = nan(n, page, hk, 2, D)
        k, v = pool[:, :, :, 0], pool[:, :, :, 1]
    elif order == "heads first":
        k, v = (nan(hk, n, page, D).permute(1, 2, 0, 3) for _ in range(2))
    else:
        k, v = (nan(n + 1, page + 2, hk + 1, D + 24)[1:, 1:page + 1, :hk, 8:8 + D] for _ in range(2))
    k.copy_(c.k)
    v.copy_(c.v)
    svq.svq_paged_attention(**a)
    b = dict(a, cache=svq.KvCache(k, v), out=torch.full_like(a["out"], 3.0), lse=torch.full_like(a["lse"], 5.0))
    svq.svq_paged_attention(**b)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    assert svq.svq_get_device_status() == svq.SVQ_OK


@pytest.mark.parametrize("order", [False, True])
def test_more_rows_than_requests(order):
    need_gpu()
    pa.check(pa.case(1, [40, 0, 900], 8, 2, 64, rows=7, order=order))


def test_empty_requests_in_stored_order():
    need_gpu()
    pa.check(pa.case(2, [0, 0], 8, 2, 64, order=True))


@pytest.mark.parametrize("in_place", [False, True])
def test_a_step_without_rows(in_place):
    """Only releases and idle requests, and no room for a row."""
    need_gpu()
    rng = np.random.default_rng(1)
    lens, new, table, free, n_free = ka.scene(rng, 30, 4, 50, 30, done=0.5, prompts=0.0)
    new = np.minimum(new, 0)
    want = oa.kv_assign(lens, new, 4, table, free, n_free, 0)
    assert want is not None
    ka.same(ka.call(lens, new, 4, table, free, n_free, 0, in_place), want)
    assert svq.svq_get_device_status() == svq.SVQ_OK


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_below_zero(interleaved):
    need_gpu()
    a = rc.case(1, 4, 4, 2, 128, 128, interleaved=interleaved)
    a["positions"][:] = torch.tensor([-1, -4096, -10 ** 8, 0], dtype=torch.int32)
    rc.check(a)


FIRST = """
import sys
sys.path.insert(0, {root!r})
import torch
from tests import test_gpu_kv_assign as ka, test_gpu_paged_attention as pa, test_gpu_rope_cache as rc
import bit_spherical_vector_b200 as svq
what = {what!r}
if what == "assign":
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    a = dict(lens=i(3), n_new=i(3) + 5, page_size=4, block_table=i(3, 3), free_pages=torch.arange(9, dtype=torch.int32, device="cuda"),
             n_free=i(1) + 9, lens_out=i(3), n_free_out=i(1), cu_rows=i(4), positions=i(20), slots=i(20))
    call, out = svq.svq_kv_assign, a["slots"]
elif what == "rope":
    a = rc.case(1, 4, 4, 2, 128, 128)
    call, out = svq.svq_qk_norm_rope_cache, a["q_out"]
else:
    a = pa.case(1, [500, 3], 8, 2, 64, order=True)
    call, out = svq.svq_paged_attention, a["out"]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    call(**a)
g.replay()
torch.cuda.synchronize()
first = out.clone()
out.zero_()
call(**a)
torch.cuda.synchronize()
assert torch.equal(out, first) and bool((first != 0).any()) and svq.svq_get_device_status() == svq.SVQ_OK
"""


@pytest.mark.parametrize("what", ["assign", "rope", "attention"])
def test_the_first_call_of_a_process_is_captured(what):
    need_gpu()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root, what=what)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
