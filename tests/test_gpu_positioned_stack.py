"""The two-layer prefill with its own norm and position rotation: the same bits as
positioning the inputs by hand, in any chunking; without it, nothing changes."""
import math

import pytest
import torch

from long_context_compressed_gated_b200 import inputs
from long_context_compressed_gated_b200.stack import stack_inputs, stack_prefill_chunked

pytestmark = pytest.mark.gpu
WL = inputs.Workload("small", T=512, H=8, d=64, m=4, k=16, W=32, HI=4, dI=64, m_hca=64, W_hca=32, seed=21)


@pytest.fixture(scope="module")
def csa():
    import long_context_compressed_gated_b200 as m
    m.lib()
    return m


def run(l1, l2, P, chunk, **kw):
    return stack_prefill_chunked(l1, l2, P, chunk, WL.m, WL.k, WL.W, WL.m_hca, WL.W_hca, return_o1=True, **kw)


@pytest.mark.parametrize("start,style,normed", [(0, 0, True), (32, 1, False)])
def test_positions_inside_the_stack(csa, start, style, normed):
    l1, l2, P = stack_inputs(WL, device="cuda")
    g = torch.Generator().manual_seed(3)
    w = dict(wq=(1 + 0.2 * torch.randn(64, generator=g)).cuda(), wk=(1 + 0.2 * torch.randn(64, generator=g)).cuda())
    position = dict(inv_freq=csa.rope_inv_freq(64 - start), rot_start=start, rot_style=style, **(w if normed else {}))
    keep = l1["Q"].clone(), l1["K"].clone(), l2["K"].clone()
    O2, O1 = run(l1, l2, P, 128, position=position)
    assert torch.equal(l1["Q"], keep[0]) and torch.equal(l1["K"], keep[1]) and torch.equal(l2["K"], keep[2])
    whole = run(l1, l2, P, 512, position=position)
    assert torch.equal(O2, whole[0]) and torch.equal(O1, whole[1])
    # by hand
    q1, k1 = csa.csa_qk_norm_rope(l1["Q"], l1["K"].unsqueeze(1), **position)
    k1 = k1.squeeze(1)
    by_hand = run(dict(l1, Q=q1, K=k1), l2, P, 512)
    assert torch.equal(O1, by_hand[1])
    q2, k2 = csa.csa_qk_norm_rope(torch.matmul(O1.view(-1, 64), P).view(512, WL.H, 64), l2["K"].unsqueeze(1), **position)
    Kc, Vc = csa.csa_compress(k2.squeeze(1), l2["V"], l2["Z"], l2["B"], WL.m_hca)
    want, _, _ = csa.hca_attn(q2, Kc, Vc, k2.squeeze(1), l2["V"], WL.m_hca, WL.W_hca, 1 / math.sqrt(64))
    assert torch.equal(O2, want)
    # positions matter, and leaving them out is what the stack did before
    plain = run(l1, l2, P, 128)
    assert not torch.equal(plain[1], O1)
    Kc, Vc = csa.csa_compress(l1["K"], l1["V"], l1["Z"], l1["B"], WL.m)
    idx, _, _ = csa.csa_indexer_topk(l1["qI_codes"], l1["qI_scales"], l1["w_codes"], l1["kI_codes"], l1["kI_scales"],
                                     WL.m, WL.k)
    want, _, _ = csa.csa_sparse_attn(l1["Q"], Kc, Vc, idx, l1["K"], l1["V"], WL.W, 1 / math.sqrt(64))
    assert torch.equal(plain[1], want)
