"""svq_qk_norm_rope_cache with the rotated queries written over the queries."""
import pytest

from tests import test_gpu_rope_cache as rc
from tests.gpu_util import need_gpu, torch

import bit_spherical_vector_b200 as svq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("M,hq,hk,dim,kv", [(1, 8, 2, 128, "f16"), (77, 13, 3, 64, "bf16"), (2048, 32, 8, 128, "bf16"),
                                            (3000, 5, 1, 256, "f16")])
def test_queries_in_place(M, hq, hk, dim, kv, interleaved):
    need_gpu()
    a = rc.case(M, M, hq, hk, dim, dim, x=kv, kv=kv, fused=False, interleaved=interleaved, pads=M // 8)
    k, v = a["cache"].k.clone(), a["cache"].v.clone()
    q = a["q"].clone()
    b = dict(a, q=q, q_out=q.view(M, hq, dim), cache=svq.KvCache(k, v))
    svq.svq_qk_norm_rope_cache(**a)
    svq.svq_qk_norm_rope_cache(**b)
    live = a["slots"] >= 0
    assert torch.equal(b["q_out"][live], a["q_out"][live]) and torch.equal(q[~live], a["q"][~live])
    assert torch.equal(k, a["cache"].k) and torch.equal(v, a["cache"].v)
