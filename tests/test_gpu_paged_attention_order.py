"""svq_paged_attention in the consumer's column order for rows of up to 65536 entries: the second kernel's two rounds
that are fetched ahead (4096 entries), the loop behind them, lines beyond 48 KB of shared memory."""
import pytest

from tests import test_gpu_paged_attention as pa
from tests.gpu_util import need_gpu, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cu", [False, True])
@pytest.mark.parametrize("hq,hk,dim,out", [(31, 31, 64, "f16"), (32, 8, 128, "bf16"), (33, 3, 128, "f16"), (64, 8, 128, "f16"),
                                           (80, 5, 256, "bf16"), (1024, 64, 64, "f16"), (256, 16, 256, "bf16")])
def test_long_rows(hq, hk, dim, out, cu):
    need_gpu()
    a = pa.case(hq + dim, [20, 0, 3], hq, hk, dim, out=out, order=True, **(dict(rows=5, cu=[0, 2, 2, 3]) if cu else {}))
    pa.check(a)


def test_long_rows_of_joined_requests():
    need_gpu()
    pa.check(pa.case(1, [3000, 5, 900], 64, 8, 128, order=True, out="bf16"))


def test_entries_sent_outside_a_long_row():
    """A column outside the row in the part that the loop handles: dropped and reported, the others in place."""
    need_gpu()
    a = pa.case(2, [20, 9], 64, 8, 128, order=True)
    whole = dict(a, out=a["out"].clone())
    pa.svq.svq_paged_attention(**whole)
    assert pa.svq.svq_get_device_status() == pa.svq.SVQ_OK
    gone = [int(a["order"][i]) for i in (4096, 8191)]
    a["order"][4096], a["order"][8191] = 8192, -1
    pa.svq.svq_paged_attention(**a)
    assert pa.svq.svq_get_device_status() == pa.svq.SVQ_ERR_INVALID_ARG
    whole["out"][:, gone] = 0
    assert torch.equal(a["out"], whole["out"])
