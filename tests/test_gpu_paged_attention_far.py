"""svq_paged_attention over a request as long as the call takes, next to 2^31 keys: four pages of keys that the
table names again and again.

Bar: a warp's share is about 90700 tiles, each with one fp32 accumulation (2 steps of 2^-23, the tensor cores may
cut) and one addition to its sum of weights (2^-24 each of two), so both are off by less than 90700 * 2^-21 = 4.4e-2
of themselves at worst; the joins and the score's own errors are far below that."""
import math

import pytest

from tests import test_gpu_paged_attention as pa
from tests.gpu_util import need_gpu, torch

import bit_spherical_vector_b200 as svq

pytestmark = pytest.mark.gpu
WIDTH, PAGE = 13106, 163855                                     # 2^31 - 18 keys


@pytest.mark.parametrize("kv", ["f16", "bf16"])
def test_the_longest_request(kv):
    need_gpu()
    dim, hq, bar = 64, 3, 90700 * 2.0 ** -21
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((4, PAGE, 1, dim), generator=g, device="cuda").to(pa.DT[kv]) for _ in range(2))
    v.copy_(v + torch.arange(4, device="cuda").view(4, 1, 1, 1))
    table = torch.randint(0, 4, (1, WIDTH), generator=g, device="cuda", dtype=torch.int32)
    cache = svq.KvCache(k, v)
    q = torch.randn((1, hq, dim), generator=g, device="cuda").to(pa.DT[kv])
    a = dict(q=q, cache=cache, lens=torch.tensor([WIDTH * PAGE], dtype=torch.int32, device="cuda"), block_table=table,
             scale=1 / math.sqrt(dim), out=torch.zeros((1, hq * dim), dtype=pa.DT[kv], device="cuda"),
             ws=pa.workspace(cache, hq), lse=torch.zeros((1, hq), device="cuda"))
    svq.svq_paged_attention(**a)
    assert svq.svq_get_device_status() == svq.SVQ_OK
    times = torch.bincount(table[0].long(), minlength=4).double()
    s = torch.einsum("hd,pkd->hpk", q[0].double(), k[:, :, 0].double()) * a["scale"]
    w = torch.exp(s - 8.0) * times[None, :, None]
    total = w.sum((1, 2))
    o = torch.einsum("hpk,pkd->hd", w, v[:, :, 0].double()) / total[:, None]
    size = torch.einsum("hpk,pkd->hd", w, v[:, :, 0].double().abs()) / total[:, None]
    eps = torch.finfo(a["out"].dtype).eps
    out = a["out"].view(hq, dim).double()
    assert bool(((out - o).abs() <= 2 * bar * size + eps / 2 * o.abs()).all())
    assert bool(((a["lse"][0].double() - torch.log(total) - 8.0).abs() <= bar + 1e-4).all())
    # an infinity that the whole range meets again and again, at the last key too
    table[0, -1] = 3
    svq.svq_paged_attention(**a)
    first = a["out"].clone()
    v[3, PAGE - 1, 0, 5] = float("-inf")
    svq.svq_paged_attention(**a)
    first.view(hq, dim)[:, 5] = float("-inf")
    assert torch.equal(a["out"], first) and svq.svq_get_device_status() == svq.SVQ_OK
