"""svq_qk_norm_rope_cache with several steps to a warp: whole and broken turns of its two-step loop, step counts
that the head counts clamp to odd ones, last slices with fewer steps or with a part of a step's heads.  Almost all
rows are padding, so the oracle has few rows to compute; the step count goes by the number of all of them."""
import pytest

from tests import test_gpu_rope_cache as rc
from tests.gpu_util import need_gpu, torch

pytestmark = pytest.mark.gpu


def steps_of(M, hq, hk, dim):
    """The launcher's rule: all steps of the call over 48 warps an SM, up to a power of two, at most 16 and at
    most what the longest kind of head has."""
    heads = 256 // dim
    q, kv = -(-hq // heads), -(-hk // heads)
    warps = torch.cuda.get_device_properties(0).multi_processor_count * 48
    want, steps = -(-M * (q + 2 * kv) // warps), 1
    while steps < want and steps < 16:
        steps *= 2
    return min(steps, max(q, kv))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("steps,M,hq,hk,dim,kw", [
    (2, 300, 32, 8, 128, dict(x="bf16", kv="bf16")),
    (3, 4000, 12, 4, 64, dict(x="f32", layout="hnd")),           # clamped, the second turn half empty
    (4, 3000, 5, 1, 256, dict(x="f16", kv="bf16")),              # two turns, then a slice of one step
    (5, 6000, 5, 1, 256, dict(x="f32", rot=112)),
    (7, 6000, 13, 3, 128, dict(x="bf16", page=24)),              # the last step has one head of two
    (8, 2048, 32, 8, 128, dict(x="bf16", kv="bf16")),
    (8, 4096, 20, 2, 128, dict(x="f32", kv="bf16", norm=False)), # slices of eight and of two steps
    (9, 5000, 33, 5, 64, dict(x="f16", rot=16)),                 # the last step has one head of four
    (16, 5000, 20, 2, 256, dict(x="f16", kv="f16", layout="both"))])
def test_steps(steps, M, hq, hk, dim, kw, interleaved):
    need_gpu()
    assert steps_of(M, hq, hk, dim) == steps
    a = rc.case(M + hq, M, hq, hk, dim, kw.get("rot", dim), interleaved=interleaved,
                **{k: v for k, v in kw.items() if k != "rot"})
    live = [0, 1, 2, M // 2, M - 2, M - 1]
    slots = a["slots"][live].clone()
    a["slots"].fill_(-1)
    a["slots"][live] = slots
    rc.check(a)
