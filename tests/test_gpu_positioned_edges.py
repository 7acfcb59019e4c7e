"""Edges of the norm + rotation, the paged append and the tree attention: refused head
dims, values that are not finite, groups that take many heads, sums over long calls."""
import math

import pytest
import torch

from tests import positioned_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def csa():
    import long_context_compressed_gated_b200 as m
    m.lib()
    return m


@pytest.mark.parametrize("d", [4, 96, 2048])
def test_backward_refuses_head_dims_without_a_workspace(csa, d):
    x = torch.zeros(3, 2, d, device="cuda")
    with pytest.raises(csa.CsaError):
        csa.csa_qk_norm_rope_backward(x, None, x, None, None)
