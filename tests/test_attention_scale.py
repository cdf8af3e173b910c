"""svq_paged_attention's scale: refused where its product with log2 e, which the kernel takes, is no number (no GPU)."""
import pytest

from tests import test_attention_abi as abi

import bit_spherical_vector_b200 as svq


@pytest.mark.parametrize("scale,status", [(2.0e38, abi.WS), (-2.0e38, abi.WS), (0.0, abi.WS), (1e-45, abi.WS),
                                          (2.4e38, abi.INV), (-2.4e38, abi.INV), (2.9e38, abi.INV), (3.4e38, abi.INV)])
def test_scale(scale, status):
    got = abi.call_attn(scale=scale)
    if status == abi.WS and got == svq.SVQ_ERR_CUDA:          # accepted, and no device to plan for
        return
    assert got == status
